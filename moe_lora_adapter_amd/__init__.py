"""MI355X-native MoE-LoRA hot path: Python binding of libmoelora.so.

The binding only marshals arguments: every step of the path runs in the HIP
kernels behind the C ABI declared in include/moe_lora.h.  PyTorch provides
device memory and the current stream.  If the library is not built the calls
raise; there is no fallback implementation.

    out = moe_lora_align(topk_ids, token_lora_mapping, E, L, block_m)
    fused_moe_lora(x, lora_a, lora_b, out, topk_weights, y,
                   mul_routed_weight=..., add_inputs=..., x_per_pair=...)

The 8-bit base side of the same layer:

    x8 = moe_lora_rms_norm_fp8(x, weight, eps=..., residual=..., y=hidden)
    moe_lora_fp8_moe_gemm(x8, w13, w13_scales, base_align, None, y, ...)
    h8 = moe_lora_silu_mul_fp8(y, h=h)
    moe_lora_fp8_moe_gemm(h8, w2, w2_scales, base_align, topk_weights, y2, ...)

The bf16 base side, from the router's logits to the layer's output:

    logits = moe_lora_gemm(x, gate, out_dtype=torch.float32)
    ids, weights = moe_lora_route(logits, topk)
    moe_lora_moe_gemm(x, w13, base_align, None, h, bias=..., delta=d13, activation="silu_mul", ...)
    moe_lora_moe_gemm(h.view(M * topk, I), w2, base_align, weights, y, mul_routed_weight=True,
                      x_per_pair=True)
    moe_lora_combine(y, topk_ids=ids, E=E, residual=x)
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoelora.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = 0, -1, -2, -3, -4
VARIANT_AUTO, VARIANT_VALU, VARIANT_MFMA = 0, 1, 2
VARIANTS = {"auto": VARIANT_AUTO, "valu": VARIANT_VALU, "mfma": VARIANT_MFMA}

# symbol -> (restype, argtypes); mirrors include/moe_lora.h
_P = ctypes.c_void_p
_I32, _I64 = ctypes.c_int32, ctypes.c_int64
SIGNATURES = {
    "moe_lora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_lora_align_capacity": (_I64, [_I64, _I32, _I32, _I32]),
    "moe_lora_align_workspace_size": (_I64, [_I64, _I32, _I32, _I32, _I32]),
    "moe_lora_align": (ctypes.c_int, [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P,
                                      _P, _P, _P, _I64, _P]),
    "moe_lora_align_noalloc": (ctypes.c_int, [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P,
                                              _P, _P, _P, _P]),
    "fused_moe_lora": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32, _I64,
                                      _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P,
                                      _I32, _P]),
    "fused_moe_lora_with_align": (ctypes.c_int, [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P,
                                                 _P, _P, _P, _P, _I32, _P, _P, _P, _I32, _I32,
                                                 _I32, _I32, _I32, _I32, _P, _I32, _P]),
    "fused_moe_lora_ws": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32,
                                         _I64, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                         _P, _I32, _P, _I64, _I32, _P]),
    "fused_moe_lora_workspace_bytes": (_I64, [_I64, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                              _I32, _I32, _I32]),
    "fused_moe_lora_variant": (ctypes.c_int, [_I64, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                              _I32, _I32, _I32]),
    "fused_moe_lora_kernel_name": (ctypes.c_char_p, [_I64, _I32, _I32, _I32, _I32, _I32, _I32,
                                                     _I32, _I32, _I32, _I32]),
    "fused_moe_lora_naive": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _I32, _I32, _I64,
                                            _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P,
                                            _I32, _P]),
    "fused_moe_lora_two_kernel_workspace_bytes": (_I64, [_I64, _I32, _I32, _I32, _I32, _I32, _I32,
                                                         _I32, _I32, _I32]),
    "fused_moe_lora_two_kernel": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _I32, _P, _I32,
                                                 _I32, _I64, _I32, _I32, _I32, _I32, _I32, _I32,
                                                 _I32, _I32, _P, _P, _I64, _P]),
    "moe_lora_accumulate": (ctypes.c_int, [_P, _P, _I64, _P]),
    "moe_lora_rms_norm_fp8": (ctypes.c_int, [_P, _P, _P, _I64, _I32, ctypes.c_float, _P, _P, _P,
                                             _P, _P]),
    "moe_lora_silu_mul_fp8": (ctypes.c_int, [_P, _I64, _I32, _P, _P, _P, _P]),
    "moe_lora_fp8_gemm": (ctypes.c_int, [_P, _P, _P, _P, _I64, _I32, _I32, _I32, _P, _P]),
    "moe_lora_fp8_moe_gemm": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P, _P, _I32, _I64,
                                             _I32, _I32, _I32, _I32, _I32, _I32, _P, _P]),
    "moe_lora_route": (ctypes.c_int, [_P, _I32, _P, _I64, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                      ctypes.c_float, _P, _P, _P]),
    "moe_lora_gemm": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P,
                                     _P]),
    "moe_lora_moe_gemm": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _I64, _I32,
                                         _I32, _I32, _I32, _I32, _I32, _I32, _P, _P]),
    "moe_lora_gemm_kernel_name": (ctypes.c_char_p, [_I64, _I32, _I32, _I32, _I32]),
    "moe_lora_moe_gemm_kernel_name": (ctypes.c_char_p, [_I64, _I32, _I32, _I32, _I32, _I32, _I32,
                                                        _I32, _I32]),
    "moe_lora_combine": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I64, _I32, _I32, _P, _P]),
}

NAIVE_MAX_PAIRS = 1024        # MOE_LORA_NAIVE_MAX_PAIRS
WITH_ALIGN_MAX_PAIRS = 64     # MOE_LORA_WITH_ALIGN_MAX_PAIRS
WITH_ALIGN_MAX_SLOTS = 64     # MOE_LORA_WITH_ALIGN_MAX_SLOTS
TWO_KERNEL_MAX_RANK = 512     # MOE_LORA_TWO_KERNEL_MAX_RANK
FP8_BLOCK = 128               # MOE_LORA_FP8_BLOCK
RMS_NORM_MAX_WIDTH = 65536    # MOE_LORA_RMS_NORM_MAX_WIDTH
ROUTE_MAX_TOPK = 64           # MOE_LORA_ROUTE_MAX_TOPK
ROUTE_MAX_EXPERTS = 1024      # MOE_LORA_ROUTE_MAX_EXPERTS
SCORINGS = {"softmax": 0, "sigmoid": 1}
ACTIVATIONS = {None: 0, "silu": 1, "gelu_tanh": 2, "silu_mul": 3, "swiglu_clamp": 4}
GATED = ("silu_mul", "swiglu_clamp")   # of gate and up: two slices in, one out


class MoeLoraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


_lib = None


def lib(path: str = LIB_PATH) -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m moe_lora_adapter_amd.build` "
                "(or __graft_entry__.build()); there is no fallback path")
        try:
            # torch's HIP runtime first: loaded behind this library's, it is a second one in the
            # process, which knows neither the other's streams nor its memory
            import torch  # noqa: F401
        except ImportError:
            pass
        handle = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().moe_lora_status_string(int(status)).decode()


def align_capacity(M: int, topk: int, E: int, block_m: int) -> int:
    v = lib().moe_lora_align_capacity(M, topk, E, block_m)
    if v < 0:
        raise MoeLoraError(v, "moe_lora_align_capacity")
    return int(v)


def align_workspace_size(M: int, topk: int, E: int, L: int, block_m: int) -> int:
    v = lib().moe_lora_align_workspace_size(M, topk, E, L, block_m)
    if v < 0:
        raise MoeLoraError(v, "moe_lora_align_workspace_size")
    return int(v)


def fused_variant(M: int, topk: int, K: int, Ns: int, S: int, E: int, L: int, r: int,
                  block_m: int, x_per_pair: bool = False, variant: str | int = "auto") -> str:
    """Name of the kernel ("valu" or "mfma") fused_moe_lora runs for these sizes."""
    v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    rc = lib().fused_moe_lora_variant(M, topk, K, Ns, S, E, L, r, block_m, int(bool(x_per_pair)),
                                      v)
    if rc < 0:
        raise MoeLoraError(rc, "fused_moe_lora_variant")
    return {VARIANT_VALU: "valu", VARIANT_MFMA: "mfma"}[rc]


def fused_kernel_name(M: int, topk: int, K: int, Ns: int, S: int, E: int, L: int, r: int,
                      block_m: int, x_per_pair: bool = False, variant: str | int = "auto") -> str:
    """Name of the GPU kernel fused_moe_lora launches for these sizes."""
    v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    args = (M, topk, K, Ns, S, E, L, r, block_m, int(bool(x_per_pair)), v)
    name = lib().fused_moe_lora_kernel_name(*args)
    if name is None:
        raise MoeLoraError(lib().fused_moe_lora_variant(*args), "fused_moe_lora_kernel_name")
    return name.decode()


@dataclass
class AlignOutput:
    sorted_token_ids: "object"        # int32 [L, cap]
    expert_ids: "object"              # int32 [L, cap // block_m]
    num_tokens_post_padded: "object"  # int32 [L]
    lora_ids: "object"                # int32 [L]
    num_active_loras: "object"        # int32 [1]
    block_m: int
    cap: int


def _dptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


_TAKEN_HERE = contextlib.nullcontext()


def _taken_on(stream):
    """Context in which a call allocates its own buffers: the allocator orders a buffer's uses by
    the stream it was taken on, which has to be the one the call writes it on."""
    if stream is None:
        return _TAKEN_HERE
    import torch
    return torch.cuda.stream(stream)


def _check(t, name, dtype, device):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def alloc_align_output(M, topk, E, L, block_m, device):
    import torch
    cap = align_capacity(M, topk, E, block_m)
    i32 = dict(dtype=torch.int32, device=device)
    return AlignOutput(torch.empty((L, cap), **i32), torch.empty((L, cap // block_m), **i32),
                       torch.empty(L, **i32), torch.empty(L, **i32), torch.empty(1, **i32),
                       block_m, cap)


def moe_lora_align(topk_ids, token_lora_mapping, E: int, L: int, block_m: int, *,
                   out: AlignOutput | None = None, workspace=None, stream=None) -> AlignOutput:
    """Group the (token, k) pairs of every LoRA slot by expert; see moe_lora.h."""
    import torch
    dev = topk_ids.device
    _check(topk_ids, "topk_ids", torch.int32, dev)
    _check(token_lora_mapping, "token_lora_mapping", torch.int32, dev)
    if topk_ids.dim() != 2 or token_lora_mapping.shape != (topk_ids.shape[0],):
        raise ValueError("topk_ids must be [M, topk] and token_lora_mapping [M]")
    M, topk = topk_ids.shape
    with _taken_on(stream):
        if out is None:
            out = alloc_align_output(M, topk, E, L, block_m, dev)
        ws_bytes = align_workspace_size(M, topk, E, L, block_m)
        if ws_bytes > 0 and workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    rc = lib().moe_lora_align(
        _dptr(topk_ids), _dptr(token_lora_mapping), M, topk, E, L, block_m,
        _dptr(out.sorted_token_ids), _dptr(out.expert_ids), _dptr(out.num_tokens_post_padded),
        _dptr(out.lora_ids), _dptr(out.num_active_loras), _dptr(workspace),
        workspace.numel() if workspace is not None else 0, _stream_ptr(stream))
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_align")
    return out


ALIGN_NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024   # MOE_LORA_ALIGN_NOALLOC_SCRATCH_BYTES


def moe_lora_align_noalloc(topk_ids, token_lora_mapping, E: int, L: int, block_m: int, *,
                           out: AlignOutput, stream=None) -> AlignOutput:
    """moe_lora_align with the library's own per-GPU scratch instead of a workspace: the
    call allocates nothing (out must be given).  Calls that may overlap on one GPU race;
    see moe_lora.h."""
    import torch
    dev = topk_ids.device
    _check(topk_ids, "topk_ids", torch.int32, dev)
    _check(token_lora_mapping, "token_lora_mapping", torch.int32, dev)
    if topk_ids.dim() != 2 or token_lora_mapping.shape != (topk_ids.shape[0],):
        raise ValueError("topk_ids must be [M, topk] and token_lora_mapping [M]")
    M, topk = topk_ids.shape
    rc = lib().moe_lora_align_noalloc(
        _dptr(topk_ids), _dptr(token_lora_mapping), M, topk, E, L, block_m,
        _dptr(out.sorted_token_ids), _dptr(out.expert_ids), _dptr(out.num_tokens_post_padded),
        _dptr(out.lora_ids), _dptr(out.num_active_loras), _stream_ptr(stream))
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_align_noalloc")
    return out


def _fused_shapes(x, lora_a, lora_b, topk_weights, y, x_per_pair):
    """Checks the tensors of a fused call; returns (M, topk, K, Ns, S, E, L, r)."""
    import torch
    dev = y.device
    _check(x, "x", torch.bfloat16, dev)
    _check(lora_a, "lora_a", torch.bfloat16, dev)
    _check(lora_b, "lora_b", torch.bfloat16, dev)
    _check(y, "y", torch.bfloat16, dev)
    if topk_weights is not None:
        _check(topk_weights, "topk_weights", torch.float32, dev)
    if lora_a.dim() != 5 or lora_b.dim() != 5 or y.dim() != 3:
        raise ValueError("lora_a [S,L,E,r,K], lora_b [S,L,E,Ns,r], y [M,topk,S*Ns]")
    S, L, E, r, K = lora_a.shape
    Ns = lora_b.shape[3]
    if tuple(lora_b.shape) != (S, L, E, Ns, r):
        raise ValueError("lora_b shape does not match lora_a")
    M, topk, N = y.shape
    if N != S * Ns:
        raise ValueError("y's last dim must be S*Ns")
    rows = M * topk if x_per_pair else M
    if tuple(x.shape) != (rows, K):
        raise ValueError(f"x must be [{rows}, {K}]")
    if topk_weights is not None and tuple(topk_weights.shape) != (M, topk):
        raise ValueError("topk_weights must be [M, topk]")
    return M, topk, K, Ns, S, E, L, r


def fused_moe_lora(x, lora_a, lora_b, align: AlignOutput, topk_weights, y, *,
                   mul_routed_weight: bool, add_inputs: bool, x_per_pair: bool = False,
                   variant: str | int = "auto", max_active_loras: int | None = None,
                   stream=None):
    """Y (+)= (X A^T) B^T per routed pair and slice, in place on y; see moe_lora.h.
    max_active_loras: host-side bound on the active slots (None: L; 0: no launch)."""
    M, topk, K, Ns, S, E, L, r = _fused_shapes(x, lora_a, lora_b, topk_weights, y, x_per_pair)
    if align.sorted_token_ids.shape[0] != L:
        raise ValueError("align output was made for another L")
    v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    rc = lib().fused_moe_lora(
        _dptr(x), int(bool(x_per_pair)), _dptr(lora_a), _dptr(lora_b),
        _dptr(align.sorted_token_ids), _dptr(align.expert_ids),
        _dptr(align.num_tokens_post_padded), L if max_active_loras is None else int(max_active_loras),
        _dptr(topk_weights),
        int(bool(mul_routed_weight)), int(bool(add_inputs)), M, topk, K, Ns, S, E, L, r,
        align.block_m, _dptr(y), v, _stream_ptr(stream))
    if rc != OK:
        raise MoeLoraError(rc, "fused_moe_lora")
    return y


def fused_moe_lora_workspace_bytes(M: int, topk: int, K: int, Ns: int, S: int, E: int, L: int,
                                   r: int, block_m: int, x_per_pair: bool = False,
                                   variant: str | int = "auto") -> int:
    """Bytes of the workspace fused_moe_lora_ws uses for these sizes (0: none)."""
    v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    n = lib().fused_moe_lora_workspace_bytes(M, topk, K, Ns, S, E, L, r, block_m,
                                             int(bool(x_per_pair)), v)
    if n < 0:
        raise MoeLoraError(int(n), "fused_moe_lora_workspace_bytes")
    return int(n)


def alloc_fused_workspace(M: int, topk: int, K: int, Ns: int, S: int, E: int, L: int, r: int,
                          block_m: int, device, x_per_pair: bool = False,
                          variant: str | int = "auto"):
    """A zero-filled workspace for fused_moe_lora_ws (at least 16 bytes)."""
    import torch
    n = fused_moe_lora_workspace_bytes(M, topk, K, Ns, S, E, L, r, block_m, x_per_pair, variant)
    return torch.zeros(max(16, n), dtype=torch.uint8, device=device)


def fused_moe_lora_ws(x, lora_a, lora_b, align: AlignOutput, topk_weights, y, *,
                      mul_routed_weight: bool, add_inputs: bool, workspace,
                      x_per_pair: bool = False, variant: str | int = "auto",
                      peer_wait: int = -1, max_active_loras: int | None = None, stream=None):
    """fused_moe_lora with a K-split workspace (zero-filled before first use); see moe_lora.h."""
    M, topk, K, Ns, S, E, L, r = _fused_shapes(x, lora_a, lora_b, topk_weights, y, x_per_pair)
    if align.sorted_token_ids.shape[0] != L:
        raise ValueError("align output was made for another L")
    v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().fused_moe_lora_ws(
        _dptr(x), int(bool(x_per_pair)), _dptr(lora_a), _dptr(lora_b),
        _dptr(align.sorted_token_ids), _dptr(align.expert_ids),
        _dptr(align.num_tokens_post_padded), L if max_active_loras is None else int(max_active_loras),
        _dptr(topk_weights),
        int(bool(mul_routed_weight)), int(bool(add_inputs)), M, topk, K, Ns, S, E, L, r,
        align.block_m, _dptr(y), v, _dptr(workspace), nbytes, int(peer_wait),
        _stream_ptr(stream))
    if rc != OK:
        raise MoeLoraError(rc, "fused_moe_lora_ws")
    return y


def fused_moe_lora_with_align(topk_ids, token_lora_mapping, x, lora_a, lora_b, topk_weights, y,
                              *, E: int, L: int, block_m: int, mul_routed_weight: bool,
                              add_inputs: bool, out: "AlignOutput | None" = None,
                              x_per_pair: bool = False, variant: str | int = "auto",
                              stream=None) -> "AlignOutput":
    """moe_lora_align and fused_moe_lora in one launch (at most WITH_ALIGN_MAX_PAIRS pairs
    and WITH_ALIGN_MAX_SLOTS slots); returns the align outputs; see moe_lora.h."""
    import torch
    M, topk, K, Ns, S, E2, L2, r = _fused_shapes(x, lora_a, lora_b, topk_weights, y, x_per_pair)
    if (E2, L2) != (E, L):
        raise ValueError("E and L must match lora_a / lora_b")
    _check(topk_ids, "topk_ids", torch.int32, y.device)
    _check(token_lora_mapping, "token_lora_mapping", torch.int32, y.device)
    if tuple(topk_ids.shape) != (M, topk) or tuple(token_lora_mapping.shape) != (M,):
        raise ValueError("topk_ids must be [M, topk] and token_lora_mapping [M]")
    if out is None:
        with _taken_on(stream):
            out = alloc_align_output(M, topk, E, L, block_m, y.device)
    rc = lib().fused_moe_lora_with_align(
        _dptr(topk_ids), _dptr(token_lora_mapping), M, topk, E, L, block_m,
        _dptr(out.sorted_token_ids), _dptr(out.expert_ids), _dptr(out.num_tokens_post_padded),
        _dptr(out.lora_ids), _dptr(out.num_active_loras), _dptr(x), int(bool(x_per_pair)),
        _dptr(lora_a), _dptr(lora_b), _dptr(topk_weights), int(bool(mul_routed_weight)),
        int(bool(add_inputs)), K, Ns, S, r, _dptr(y),
        VARIANTS[variant] if isinstance(variant, str) else int(variant), _stream_ptr(stream))
    if rc != OK:
        raise MoeLoraError(rc, "fused_moe_lora_with_align")
    return out


def fused_moe_lora_naive(x, lora_a, lora_b, topk_ids, token_lora_mapping, topk_weights, y, *,
                         mul_routed_weight: bool, add_inputs: bool, block_m: int = 16,
                         x_per_pair: bool = False, variant: str | int = "auto", stream=None):
    """fused_moe_lora without the align step (M * topk <= NAIVE_MAX_PAIRS); see moe_lora.h."""
    import torch
    M, topk, K, Ns, S, E, L, r = _fused_shapes(x, lora_a, lora_b, topk_weights, y, x_per_pair)
    _check(topk_ids, "topk_ids", torch.int32, y.device)
    _check(token_lora_mapping, "token_lora_mapping", torch.int32, y.device)
    if tuple(topk_ids.shape) != (M, topk) or tuple(token_lora_mapping.shape) != (M,):
        raise ValueError("topk_ids must be [M, topk] and token_lora_mapping [M]")
    rc = lib().fused_moe_lora_naive(
        _dptr(x), int(bool(x_per_pair)), _dptr(lora_a), _dptr(lora_b), _dptr(topk_ids),
        _dptr(token_lora_mapping), _dptr(topk_weights), int(bool(mul_routed_weight)),
        int(bool(add_inputs)), M, topk, K, Ns, S, E, L, r, block_m, _dptr(y),
        VARIANTS[variant] if isinstance(variant, str) else int(variant), _stream_ptr(stream))
    if rc != OK:
        raise MoeLoraError(rc, "fused_moe_lora_naive")
    return y


def two_kernel_workspace_bytes(M: int, topk: int, K: int, Ns: int, S: int, E: int, L: int, r: int,
                               block_m: int, x_per_pair: bool = False) -> int:
    v = lib().fused_moe_lora_two_kernel_workspace_bytes(M, topk, K, Ns, S, E, L, r, block_m,
                                                        int(bool(x_per_pair)))
    if v < 0:
        raise MoeLoraError(v, "fused_moe_lora_two_kernel_workspace_bytes")
    return int(v)


def fused_moe_lora_two_kernel(x, lora_a, lora_b, align: AlignOutput, topk_weights, y, *,
                              mul_routed_weight: bool, add_inputs: bool, x_per_pair: bool = False,
                              workspace=None, max_active_loras: int | None = None, stream=None):
    """fused_moe_lora as shrink + expand with the rank vectors in `workspace` (ranks up to
    TWO_KERNEL_MAX_RANK); see moe_lora.h."""
    import torch
    M, topk, K, Ns, S, E, L, r = _fused_shapes(x, lora_a, lora_b, topk_weights, y, x_per_pair)
    if align.sorted_token_ids.shape[0] != L:
        raise ValueError("align output was made for another L")
    nbytes = two_kernel_workspace_bytes(M, topk, K, Ns, S, E, L, r, align.block_m, x_per_pair)
    if workspace is None:
        with _taken_on(stream):
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=y.device)
    _check(workspace, "workspace", workspace.dtype, y.device)
    rc = lib().fused_moe_lora_two_kernel(
        _dptr(x), int(bool(x_per_pair)), _dptr(lora_a), _dptr(lora_b),
        _dptr(align.sorted_token_ids), _dptr(align.expert_ids),
        _dptr(align.num_tokens_post_padded), L if max_active_loras is None else int(max_active_loras),
        _dptr(topk_weights),
        int(bool(mul_routed_weight)), int(bool(add_inputs)), M, topk, K, Ns, S, E, L, r,
        align.block_m, _dptr(y), _dptr(workspace), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    if rc != OK:
        raise MoeLoraError(rc, "fused_moe_lora_two_kernel")
    return y


def moe_lora_accumulate(y, delta, stream=None):
    """y += delta (bf16, elementwise, one rounding): the join of the dual-stream path; see
    moe_lora.h.  Ordering the two streams is the caller's."""
    import torch
    _check(y, "y", torch.bfloat16, y.device)
    _check(delta, "delta", torch.bfloat16, y.device)
    if y.numel() != delta.numel():
        raise ValueError("y and delta must have the same number of elements")
    rc = lib().moe_lora_accumulate(_dptr(y), _dptr(delta), y.numel(), _stream_ptr(stream))
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_accumulate")
    return y


@dataclass
class Fp8Rows:
    """8-bit rows: a value is q * scale of its row and block of 128 columns."""
    q: "object"        # float8_e4m3fn [M, K]
    scales: "object"   # float32 [ceil(K / 128), M]


def fp8_blocks(n: int) -> int:
    """Scale blocks of n columns."""
    return -(-n // FP8_BLOCK)


def alloc_fp8_rows(M: int, K: int, device) -> Fp8Rows:
    import torch
    return Fp8Rows(torch.empty((M, K), dtype=torch.float8_e4m3fn, device=device),
                   torch.empty((fp8_blocks(K), M), dtype=torch.float32, device=device))


def _refuse(t, name, dtype, device, shape):
    """Raise for a tensor that is not contiguous, of this type and shape, on this device."""
    _check(t, name, dtype, device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _call(name, x, stream, *args):
    """Call an entry point on x's device: its stream last, that device current."""
    import torch
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"{name} needs tensors on a GPU, got {device}")
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    with torch.cuda.device(device):
        raw = torch.cuda.current_stream() if stream is None else stream
        rc = getattr(lib(), name)(*args, raw.cuda_stream)
    if rc != OK:
        raise MoeLoraError(rc, name)


def _direct(torch, device, stream):
    """The raw current stream when nothing has to be switched for a call on `device`, else None:
    making a Stream object costs more than the call.  The two names are not torch's public ones;
    where they are missing the calls go through _call."""
    if stream is None and device >= 0:
        try:
            if torch._C._cuda_getDevice() == device:
                return torch._C._cuda_getCurrentRawStream(device)
        except AttributeError:
            pass
    return None


# The checks below are written out, attribute by attribute: in a serving loop's small calls a
# helper per tensor costs as much as the launch.

def moe_lora_rms_norm_fp8(x, weight, *, eps: float = 1e-6, residual=None, residual_out=None, y=None,
                          out: Fp8Rows | None = None, stream=None) -> Fp8Rows:
    """RMS norm of x (+ residual) as 8-bit rows, and as bf16 in y when given; the sum goes to
    residual_out (None: in place on residual); see moe_lora.h.  Buffers that a call allocates are
    of the stream it runs on."""
    import torch
    bf = torch.bfloat16
    if not isinstance(x, torch.Tensor) or x.dtype is not bf or not x.is_contiguous():
        _check(x, "x", bf, x.device)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [M, H]")
    M, H = shape
    at = x.get_device()
    if out is None:
        with _taken_on(stream):
            out = alloc_fp8_rows(M, H, x.device)
    if (weight.dtype is not bf or weight.shape != (H,) or not weight.is_contiguous()
            or weight.get_device() != at):
        _refuse(weight, "weight", bf, x.device, (H,))
    pr = po = py = None
    if residual is not None:
        if (residual.dtype is not bf or residual.shape != shape or not residual.is_contiguous()
                or residual.get_device() != at):
            _refuse(residual, "residual", bf, x.device, shape)
        pr = po = residual.data_ptr()
        if residual_out is not None:
            if (residual_out.dtype is not bf or residual_out.shape != shape
                    or not residual_out.is_contiguous() or residual_out.get_device() != at):
                _refuse(residual_out, "residual_out", bf, x.device, shape)
            po = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if y is not None:
        if (y.dtype is not bf or y.shape != shape or not y.is_contiguous()
                or y.get_device() != at):
            _refuse(y, "y", bf, x.device, shape)
        py = y.data_ptr()
    pq, ps = _rows_ptrs(torch, out, "out", M, H, x, at)
    raw = _direct(torch, at, stream)
    if raw is None:
        _call("moe_lora_rms_norm_fp8", x, stream, x.data_ptr(), pr, weight.data_ptr(), M, H, eps,
              po, py, pq, ps)
        return out
    rc = lib().moe_lora_rms_norm_fp8(x.data_ptr(), pr, weight.data_ptr(), M, H, eps, po, py, pq,
                                     ps, raw)
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_rms_norm_fp8")
    return out


def _rows_ptrs(torch, rows, name, M, K, like, at):
    """Checks 8-bit rows [M, K] on the device of `like`; their two addresses."""
    q, s = rows.q, rows.scales
    if (q.dtype is not torch.float8_e4m3fn or q.shape != (M, K) or not q.is_contiguous()
            or q.get_device() != at):
        _refuse(q, name + ".q", torch.float8_e4m3fn, like.device, (M, K))
    kb = -(-K // FP8_BLOCK)
    if (s.dtype is not torch.float32 or s.shape != (kb, M) or not s.is_contiguous()
            or s.get_device() != at):
        _refuse(s, name + ".scales", torch.float32, like.device, (kb, M))
    return q.data_ptr(), s.data_ptr()


def moe_lora_silu_mul_fp8(y, *, h=None, out: Fp8Rows | None = None, stream=None) -> Fp8Rows:
    """silu(gate) * up of y = [..., gate | up] as 8-bit rows, and as bf16 in h when given; see
    moe_lora.h."""
    import torch
    bf = torch.bfloat16
    if not isinstance(y, torch.Tensor) or y.dtype is not bf or not y.is_contiguous():
        _check(y, "y", bf, y.device)
    shape = y.shape
    if len(shape) < 2 or shape[-1] % 2:
        raise ValueError("y must be [..., 2 * I]")
    I = shape[-1] // 2
    P = y.numel() // (2 * I) if I else 0
    at, ph = y.get_device(), None
    if h is not None:
        if (h.dtype is not bf or h.shape != (P, I) or not h.is_contiguous()
                or h.get_device() != at):
            _refuse(h, "h", bf, y.device, (P, I))
        ph = h.data_ptr()
    if out is None:
        with _taken_on(stream):
            out = alloc_fp8_rows(P, I, y.device)
    pq, ps = _rows_ptrs(torch, out, "out", P, I, y, at)
    raw = _direct(torch, at, stream)
    if raw is None:
        _call("moe_lora_silu_mul_fp8", y, stream, y.data_ptr(), P, I, ph, pq, ps)
        return out
    rc = lib().moe_lora_silu_mul_fp8(y.data_ptr(), P, I, ph, pq, ps, raw)
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_silu_mul_fp8")
    return out


def _weight_ptrs(torch, w, w_scales, shape, at):
    """Checks 8-bit weights [..., Ns, K] and their scales; their two addresses."""
    if w.dtype is not torch.float8_e4m3fn or not w.is_contiguous():
        _check(w, "w", torch.float8_e4m3fn, w.device)
    want = (*shape[:-2], -(-shape[-2] // FP8_BLOCK), -(-shape[-1] // FP8_BLOCK))
    if (w_scales.dtype is not torch.float32 or w_scales.shape != want
            or not w_scales.is_contiguous() or w_scales.get_device() != at):
        _refuse(w_scales, "w_scales", torch.float32, w.device, want)
    return w.data_ptr(), w_scales.data_ptr()


def moe_lora_fp8_gemm(x: Fp8Rows, w, w_scales, y=None, *, stream=None):
    """8-bit rows times w [S, Ns, K] (e4m3, a scale per 128 x 128 block of a slice); y bf16
    [M, S*Ns] is allocated when not given; see moe_lora.h."""
    import torch
    shape, at = w.shape, w.get_device()
    if len(shape) != 3 or x.q.dim() != 2:
        raise ValueError("w must be [S, Ns, K] and x.q [M, K]")
    S, Ns, K = shape
    M = x.q.shape[0]
    pw, pws = _weight_ptrs(torch, w, w_scales, shape, at)
    pq, ps = _rows_ptrs(torch, x, "x", M, K, w, at)
    if y is None:
        with _taken_on(stream):
            y = torch.empty((M, S * Ns), dtype=torch.bfloat16, device=w.device)
    elif (y.dtype is not torch.bfloat16 or y.shape != (M, S * Ns) or not y.is_contiguous()
          or y.get_device() != at):
        _refuse(y, "y", torch.bfloat16, w.device, (M, S * Ns))
    raw = _direct(torch, at, stream)
    if raw is None:
        _call("moe_lora_fp8_gemm", w, stream, pq, ps, pw, pws, M, K, Ns, S, y.data_ptr())
        return y
    rc = lib().moe_lora_fp8_gemm(pq, ps, pw, pws, M, K, Ns, S, y.data_ptr(), raw)
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_fp8_gemm")
    return y


def moe_lora_fp8_moe_gemm(x: Fp8Rows, w, w_scales, align: AlignOutput, topk_weights, y, *,
                          mul_routed_weight: bool, x_per_pair: bool = False, stream=None):
    """8-bit rows times each routed pair's expert of w [E, S, Ns, K], into y [M, topk, S*Ns]; align
    is one slot's (L = 1); see moe_lora.h."""
    import torch
    i32, shape, at = torch.int32, w.shape, w.get_device()
    if len(shape) != 4 or y.dim() != 3 or x.q.dim() != 2:
        raise ValueError("w must be [E, S, Ns, K], y [M, topk, S*Ns] and x.q [rows, K]")
    E, S, Ns, K = shape
    M, topk, N = y.shape
    if N != S * Ns:
        raise ValueError("y's last dim must be S*Ns")
    if y.dtype is not torch.bfloat16 or not y.is_contiguous() or y.get_device() != at:
        _check(y, "y", torch.bfloat16, w.device)
    pw, pws = _weight_ptrs(torch, w, w_scales, shape, at)
    pq, ps = _rows_ptrs(torch, x, "x", M * topk if x_per_pair else M, K, w, at)
    ptw = None
    if topk_weights is not None:
        if (topk_weights.dtype is not torch.float32 or topk_weights.shape != (M, topk)
                or not topk_weights.is_contiguous() or topk_weights.get_device() != at):
            _refuse(topk_weights, "topk_weights", torch.float32, w.device, (M, topk))
        ptw = topk_weights.data_ptr()
    block_m = align.block_m
    cap = align_capacity(M, topk, E, block_m)
    ids, eids, ntpp = align.sorted_token_ids, align.expert_ids, align.num_tokens_post_padded
    for t, name, want in ((ids, "sorted_token_ids", (1, cap)),
                          (eids, "expert_ids", (1, cap // block_m)),
                          (ntpp, "num_tokens_post_padded", (1,))):
        if t.dtype is not i32 or t.shape != want or not t.is_contiguous() or t.get_device() != at:
            _refuse(t, "align." + name, i32, w.device, want)
    args = (pq, ps, 1 if x_per_pair else 0, pw, pws, ids.data_ptr(), eids.data_ptr(),
            ntpp.data_ptr(), ptw, 1 if mul_routed_weight else 0, M, topk, K, Ns, S, E, block_m,
            y.data_ptr())
    raw = _direct(torch, at, stream)
    if raw is None:
        _call("moe_lora_fp8_moe_gemm", w, stream, *args)
        return y
    rc = lib().moe_lora_fp8_moe_gemm(*args, raw)
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_fp8_moe_gemm")
    return y


def _align_ptrs(torch, align, M, topk, E, like, at):
    """Checks one slot's align outputs on the device of `like`; their three addresses."""
    i32, block_m = torch.int32, align.block_m
    cap = align_capacity(M, topk, E, block_m)
    ids, eids, ntpp = align.sorted_token_ids, align.expert_ids, align.num_tokens_post_padded
    for t, name, want in ((ids, "sorted_token_ids", (1, cap)),
                          (eids, "expert_ids", (1, cap // block_m)),
                          (ntpp, "num_tokens_post_padded", (1,))):
        if t.dtype is not i32 or t.shape != want or not t.is_contiguous() or t.get_device() != at:
            _refuse(t, "align." + name, i32, like.device, want)
    return ids.data_ptr(), eids.data_ptr(), ntpp.data_ptr()


def _activation(name):
    """Number of an activation, and whether it takes gate and up."""
    try:
        return ACTIVATIONS[name], name in GATED
    except KeyError:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {name!r}") from None


def _optional(t, name, dtype, shape, like, at):
    """Address of a tensor that may be None, checked."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != at):
        _refuse(t, name, dtype, like.device, shape)
    return t.data_ptr()


def _in_32_bits(bits, where):
    """Refuses sizes, given or-ed together, that a call's 32-bit arguments would cut short."""
    if bits >> 31 > 0:
        raise MoeLoraError(ERR_UNSUPPORTED, where)


def moe_lora_route(logits, topk: int, *, scoring: str = "softmax", bias=None, n_group: int = 1,
                   topk_group: int = 1, group_top: int = 1, renormalize: bool = True,
                   scale: float = 1.0, topk_ids=None, topk_weights=None, stream=None):
    """Experts and weights of every row of logits [M, E] (fp32 or bf16): (topk_ids int32,
    topk_weights fp32), both [M, topk], allocated when not given; -1 and 0 where no expert is
    left; see moe_lora.h."""
    import torch
    bf16 = isinstance(logits, torch.Tensor) and logits.dtype is torch.bfloat16
    if not bf16:
        _check(logits, "logits", torch.float32, getattr(logits, "device", None))
    elif not logits.is_contiguous():
        _check(logits, "logits", torch.bfloat16, logits.device)
    if logits.dim() != 2:
        raise ValueError("logits must be [M, E]")
    if scoring not in SCORINGS:
        raise ValueError(f"scoring must be one of {list(SCORINGS)}, got {scoring!r}")
    M, E = logits.shape
    _in_32_bits(E | topk | n_group | topk_group | group_top, "moe_lora_route")
    at, want = logits.get_device(), (M, topk)
    pb = _optional(bias, "bias", torch.float32, (E,), logits, at)
    if topk_ids is None or topk_weights is None:
        if topk < 1:
            raise MoeLoraError(ERR_INVALID, "moe_lora_route")
        with _taken_on(stream):
            if topk_ids is None:
                topk_ids = torch.empty(want, dtype=torch.int32, device=logits.device)
            if topk_weights is None:
                topk_weights = torch.empty(want, dtype=torch.float32, device=logits.device)
    pi = _optional(topk_ids, "topk_ids", torch.int32, want, logits, at)
    pw = _optional(topk_weights, "topk_weights", torch.float32, want, logits, at)
    args = (logits.data_ptr(), 1 if bf16 else 0, pb, M, E, topk, SCORINGS[scoring], n_group,
            topk_group, group_top, 1 if renormalize else 0, scale, pi, pw)
    raw = _direct(torch, at, stream)
    if raw is None:
        _call("moe_lora_route", logits, stream, *args)
        return topk_ids, topk_weights
    rc = lib().moe_lora_route(*args, raw)
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_route")
    return topk_ids, topk_weights


def moe_lora_gemm(x, w, y=None, *, bias=None, delta=None, activation: str | None = None,
                  residual=None, out_dtype=None, stream=None):
    """activation(x w^T + bias + delta) + residual for w [S, Ns, K]; y [M, S*Ns] ([M, Ns] with a
    gated activation) is bf16 or fp32, allocated as out_dtype (None: bf16) when not given; see
    moe_lora.h."""
    import torch
    bf = torch.bfloat16
    if not isinstance(w, torch.Tensor) or w.dtype is not bf or not w.is_contiguous():
        _check(w, "w", bf, getattr(w, "device", None))
    if w.dim() != 3 or x.dim() != 2:
        raise ValueError("w must be [S, Ns, K] and x [M, K]")
    S, Ns, K = w.shape
    _in_32_bits(S | Ns | K, "moe_lora_gemm")
    M, at, N = x.shape[0], w.get_device(), S * Ns
    act, gated = _activation(activation)
    No = Ns if gated else N
    if x.dtype is not bf or x.shape != (M, K) or not x.is_contiguous() or x.get_device() != at:
        _refuse(x, "x", bf, w.device, (M, K))
    pb = _optional(bias, "bias", bf, (N,), w, at) if bias is not None else None
    pd = _optional(delta, "delta", bf, (M, N), w, at) if delta is not None else None
    pr = _optional(residual, "residual", bf, (M, No), w, at) if residual is not None else None
    if y is None:
        with _taken_on(stream):
            y = torch.empty((M, No), dtype=bf if out_dtype is None else out_dtype, device=w.device)
    elif out_dtype is not None and y.dtype is not out_dtype:
        raise TypeError(f"y must be {out_dtype}, got {y.dtype}")
    wide = y.dtype is torch.float32
    if ((y.dtype is not bf and not wide) or y.shape != (M, No) or not y.is_contiguous()
            or y.get_device() != at):
        _refuse(y, "y", bf, w.device, (M, No))
    args = (x.data_ptr(), w.data_ptr(), pb, pd, pr, M, K, Ns, S, act, 1 if wide else 0,
            y.data_ptr())
    raw = _direct(torch, at, stream)
    if raw is None:
        _call("moe_lora_gemm", w, stream, *args)
        return y
    rc = lib().moe_lora_gemm(*args, raw)
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_gemm")
    return y


def moe_lora_moe_gemm(x, w, align: AlignOutput, topk_weights, y, *, mul_routed_weight: bool,
                      x_per_pair: bool = False, bias=None, delta=None,
                      activation: str | None = None, stream=None):
    """moe_lora_gemm with each routed pair's expert of w [E, S, Ns, K] and its bias [E, S*Ns], the
    routed weight before delta [M, topk, S*Ns] (zeros where the adapters wrote nothing), into y [M, topk, S*Ns] ([M, topk, Ns] with a gated
    activation); align is one slot's (L = 1); see moe_lora.h."""
    import torch
    bf = torch.bfloat16
    if not isinstance(w, torch.Tensor) or w.dtype is not bf or not w.is_contiguous():
        _check(w, "w", bf, getattr(w, "device", None))
    if w.dim() != 4 or y.dim() != 3 or x.dim() != 2:
        raise ValueError("w must be [E, S, Ns, K], y [M, topk, N] and x [rows, K]")
    E, S, Ns, K = w.shape
    at, N = w.get_device(), S * Ns
    act, gated = _activation(activation)
    M, topk, No = y.shape
    _in_32_bits(E | S | Ns | K | topk, "moe_lora_moe_gemm")
    if No != (Ns if gated else N):
        raise ValueError(f"y's last dim must be {Ns if gated else N}, got {No}")
    if y.dtype is not bf or not y.is_contiguous() or y.get_device() != at:
        _check(y, "y", bf, w.device)
    rows = M * topk if x_per_pair else M
    if x.dtype is not bf or x.shape != (rows, K) or not x.is_contiguous() or x.get_device() != at:
        _refuse(x, "x", bf, w.device, (rows, K))
    pb = _optional(bias, "bias", bf, (E, N), w, at) if bias is not None else None
    pd = _optional(delta, "delta", bf, (M, topk, N), w, at) if delta is not None else None
    ptw = None
    if topk_weights is not None:
        ptw = _optional(topk_weights, "topk_weights", torch.float32, (M, topk), w, at)
    pids, peids, pntpp = _align_ptrs(torch, align, M, topk, E, w, at)
    args = (x.data_ptr(), 1 if x_per_pair else 0, w.data_ptr(), pb, pd, pids, peids, pntpp, ptw,
            1 if mul_routed_weight else 0, M, topk, K, Ns, S, E, align.block_m, act, y.data_ptr())
    raw = _direct(torch, at, stream)
    if raw is None:
        _call("moe_lora_moe_gemm", w, stream, *args)
        return y
    rc = lib().moe_lora_moe_gemm(*args, raw)
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_moe_gemm")
    return y


def gemm_kernel_name(M: int, K: int, Ns: int, S: int, activation: str | None = None) -> str:
    """Name and tile of the GPU kernel moe_lora_gemm launches for these sizes."""
    name = lib().moe_lora_gemm_kernel_name(M, K, Ns, S, _activation(activation)[0])
    if name is None:
        raise MoeLoraError(ERR_INVALID, "moe_lora_gemm_kernel_name")
    return name.decode()


def moe_gemm_kernel_name(M: int, topk: int, K: int, Ns: int, S: int, E: int, block_m: int,
                         x_per_pair: bool = False, activation: str | None = None) -> str:
    """Name and tile of the GPU kernel moe_lora_moe_gemm launches for these sizes."""
    name = lib().moe_lora_moe_gemm_kernel_name(M, topk, K, Ns, S, E, block_m,
                                               int(bool(x_per_pair)), _activation(activation)[0])
    if name is None:
        raise MoeLoraError(ERR_INVALID, "moe_lora_moe_gemm_kernel_name")
    return name.decode()


def moe_lora_combine(y, out=None, *, topk_weights=None, topk_ids=None, E: int | None = None,
                     residual=None, stream=None):
    """sum over k of y [M, topk, N] (times topk_weights) + residual, into out [M, N] (allocated when
    not given); with topk_ids, pairs whose id is outside [0, E) are left out; see moe_lora.h."""
    import torch
    bf = torch.bfloat16
    if not isinstance(y, torch.Tensor) or y.dtype is not bf or not y.is_contiguous():
        _check(y, "y", bf, getattr(y, "device", None))
    if y.dim() != 3:
        raise ValueError("y must be [M, topk, N]")
    if topk_ids is not None and E is None:
        raise ValueError("topk_ids needs E, the number of experts here")
    M, topk, N = y.shape
    E = E or 0
    _in_32_bits(topk | N | E, "moe_lora_combine")
    at = y.get_device()
    pw = _optional(topk_weights, "topk_weights", torch.float32, (M, topk), y, at)
    pi = _optional(topk_ids, "topk_ids", torch.int32, (M, topk), y, at)
    pr = _optional(residual, "residual", bf, (M, N), y, at)
    if out is None:
        with _taken_on(stream):
            out = torch.empty((M, N), dtype=bf, device=y.device)
    po = _optional(out, "out", bf, (M, N), y, at)
    args = (y.data_ptr(), pw, pi, E, pr, M, topk, N, po)
    raw = _direct(torch, at, stream)
    if raw is None:
        _call("moe_lora_combine", y, stream, *args)
        return out
    rc = lib().moe_lora_combine(*args, raw)
    if rc != OK:
        raise MoeLoraError(rc, "moe_lora_combine")
    return out
