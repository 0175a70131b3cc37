"""FP8 E4M3 (ASH + DS) compression of tensor-parallel tensors on MI355X (gfx950).

Thin binding of the C ABI in ``include/tfp8.h`` (``libtfp8.so``, built in this directory by
``build.py``).  This module only marshals arguments: PyTorch supplies device memory and the
current HIP stream, and every step of compress, decompress, the reduce and the accumulation runs
in the library's kernels.  There is no CPU path: without the built library, or for tensors not
on a GPU, the calls raise.

Method: page "TACO: Efficient Communication Compression of Intermediate Tensors for Scalable
Tensor-Parallel LLM Training" (section 2.B.1-2.B.2); local reduce and gradient accumulation:
page "AGoQ: Activation and Gradient Quantization for Memory-Efficient Distributed Training of
LLMs" (section 2.B).
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "compress", "decompress", "reduce_fp8", "compress_raw", "decompress_raw", "reduce_fp8_raw",
    "status_string", "lib", "LIB_PATH", "TFP8Error", "BF16", "F32", "SUPPORTED_BLOCKS",
    "FLAG_INT8", "FLAG_NO_ROTATION", "accumulate", "accumulate_raw", "reduce_strided_raw",
    "compress_t", "matmul", "matmul_grouped", "matmul_grouped_t", "padded_rows",
    "compress_t_raw", "matmul_raw", "matmul_grouped_raw", "matmul_grouped_t_raw",
    "PRODUCT_BLOCKS", "MAX_GROUPS",
    "grad_norm", "adamw", "adamw_state", "grad_norm_raw", "adamw_raw",
    "moe_layer", "moe_layer_raw", "MOE_TOKENS", "MOE_EXPERTS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtfp8.so")
BF16, F32 = 0, 1
FLAG_INT8, FLAG_NO_ROTATION = 1, 2  # variant flags of the *_ex entry points (include/tfp8.h)
SUPPORTED_BLOCKS = (64, 128, 256, 512)
PRODUCT_BLOCKS = (128, 256, 512)  # blocks that the products of compressed operands take
MAX_GROUPS = 65536
MOE_TOKENS, MOE_EXPERTS = 64, 512  # the most that moe_layer takes
_MOE_ALL_EXPERTS = 4  # TFP8_MOE_ALL_EXPERTS (include/tfp8.h)

_STATUS = {0: "TFP8_OK", -1: "TFP8_E_NULL", -2: "TFP8_E_SIZE", -3: "TFP8_E_BLOCK",
           -4: "TFP8_E_DTYPE", -5: "TFP8_E_ALIGN", -6: "TFP8_E_ARG", -7: "TFP8_E_HIP"}


class TFP8Error(RuntimeError):
    """A status other than TFP8_OK; ``.status`` holds the code."""

    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def _declare(L: ctypes.CDLL) -> ctypes.CDLL:
    """Argument and result types of the C ABI's entry points on an opened build of the library."""
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    L.tfp8_compress.argtypes = [vp, i32, i64, i32, f32, vp, vp, vp, vp]
    L.tfp8_compress.restype = i32
    L.tfp8_decompress.argtypes = [vp, vp, vp, i64, i32, vp, i32, vp]
    L.tfp8_decompress.restype = i32
    L.tfp8_reduce_fp8.argtypes = [vp, vp, vp, i32, i64, i32, f32, vp, vp, vp, vp]
    L.tfp8_reduce_fp8.restype = i32
    u32 = ctypes.c_uint32
    L.tfp8_compress_ex.argtypes = [vp, i32, i64, i32, f32, u32, vp, vp, vp, vp]
    L.tfp8_compress_ex.restype = i32
    L.tfp8_decompress_ex.argtypes = [vp, vp, vp, i64, i32, u32, vp, i32, vp]
    L.tfp8_decompress_ex.restype = i32
    L.tfp8_reduce_ex.argtypes = [vp, vp, vp, i32, i64, i32, f32, u32, vp, vp, vp, vp]
    L.tfp8_reduce_ex.restype = i32
    L.tfp8_reduce_strided.argtypes = [vp, i64, vp, i64, vp, i64, i32, i64, i32, f32, u32,
                                      vp, vp, vp, vp]
    L.tfp8_reduce_strided.restype = i32
    L.tfp8_accumulate.argtypes = [vp, vp, vp, vp, i32, i64, i32, f32, u32, vp, vp, vp, vp]
    L.tfp8_accumulate.restype = i32
    L.tfp8_padded_rows.argtypes = [i64, i32, i32]
    L.tfp8_padded_rows.restype = i64
    L.tfp8_compress_t.argtypes = [vp, i32, i64, i64, i64, vp, i32, i32, f32, u32, vp, vp, vp, vp]
    L.tfp8_compress_t.restype = i32
    operand = [vp, i64, vp, vp, i64]
    L.tfp8_matmul.argtypes = [*operand, *operand, i64, i64, i64, i32, vp, i32, i64, vp]
    L.tfp8_matmul.restype = i32
    L.tfp8_matmul_grouped.argtypes = [*operand, *operand, vp, i32, i64, i64, i64, i32, vp, i32,
                                      i64, vp]
    L.tfp8_matmul_grouped.restype = i32
    L.tfp8_matmul_grouped_t.argtypes = [*operand, *operand, vp, i32, i64, i64, i64, i32, vp, i32,
                                        vp]
    L.tfp8_matmul_grouped_t.restype = i32
    L.tfp8_grad_norm_workspace.argtypes = [i32]
    L.tfp8_grad_norm_workspace.restype = i64
    L.tfp8_grad_norm.argtypes = [vp, i32, i32, f32, vp, i64, vp, vp, vp]
    L.tfp8_grad_norm.restype = i32
    L.tfp8_adamw.argtypes = [vp, i32, i32, i32, *[vp] * 8, i64, vp, vp]
    L.tfp8_adamw.restype = i32
    L.tfp8_moe_workspace.argtypes = [i64] * 5
    L.tfp8_moe_workspace.restype = i64
    L.tfp8_moe_layer.argtypes = [vp, i32, i64, vp, i32, *[vp] * 6, *[i64] * 5, i32, u32, vp, i64, vp,
                                 i32, i64, vp]
    L.tfp8_moe_layer.restype = i32
    L.tfp8_status_string.argtypes = [i32]
    L.tfp8_status_string.restype = ctypes.c_char_p
    L.tfp8_version.argtypes = []
    L.tfp8_version.restype = i32
    return L


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run fp8_compression_tensor_amd/build.py "
                               "(or __graft_entry__.build())")
        _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def status_string(status: int) -> str:
    return lib().tfp8_status_string(int(status)).decode()


def _check(status: int):
    if status != 0:
        raise TFP8Error(status, status_string(status))


# ---------------------------------------------------------------------------------- raw calls
# Pointers are integers (device addresses); `stream` is a raw hipStream_t (0 = default stream).

def compress_raw(x_ptr: int, x_dtype: int, n: int, block: int, target: float, codes_ptr: int,
                 alpha_ptr: int, scale_ptr: int, stream: int = 0, flags: int = 0) -> int:
    if flags:
        return lib().tfp8_compress_ex(x_ptr, x_dtype, n, block, target, flags, codes_ptr,
                                      alpha_ptr, scale_ptr, stream)
    return lib().tfp8_compress(x_ptr, x_dtype, n, block, target, codes_ptr, alpha_ptr,
                               scale_ptr, stream)


def decompress_raw(codes_ptr: int, alpha_ptr: int, scale_ptr: int, n: int, block: int,
                   out_ptr: int, out_dtype: int, stream: int = 0, flags: int = 0) -> int:
    if flags:
        return lib().tfp8_decompress_ex(codes_ptr, alpha_ptr, scale_ptr, n, block, flags, out_ptr,
                                        out_dtype, stream)
    return lib().tfp8_decompress(codes_ptr, alpha_ptr, scale_ptr, n, block, out_ptr, out_dtype,
                                 stream)


def reduce_fp8_raw(codes_ptr: int, alpha_ptr: int, scale_ptr: int, P: int, n: int, block: int,
                   target: float, codes_out_ptr: int, alpha_out_ptr: int, scale_out_ptr: int,
                   stream: int = 0, flags: int = 0) -> int:
    if flags:
        return lib().tfp8_reduce_ex(codes_ptr, alpha_ptr, scale_ptr, P, n, block, target, flags,
                                    codes_out_ptr, alpha_out_ptr, scale_out_ptr, stream)
    return lib().tfp8_reduce_fp8(codes_ptr, alpha_ptr, scale_ptr, P, n, block, target,
                                 codes_out_ptr, alpha_out_ptr, scale_out_ptr, stream)


def reduce_strided_raw(codes_ptr: int, codes_stride: int, alpha_ptr: int, alpha_stride: int,
                       scale_ptr: int, scale_stride: int, P: int, n: int, block: int,
                       target: float, codes_out_ptr: int, alpha_out_ptr: int, scale_out_ptr: int,
                       stream: int = 0, flags: int = 0) -> int:
    """Contribution p at codes_ptr + p * codes_stride (bytes), alpha_ptr / scale_ptr + p times
    their stride (float32 elements)."""
    return lib().tfp8_reduce_strided(codes_ptr, codes_stride, alpha_ptr, alpha_stride, scale_ptr,
                                     scale_stride, P, n, block, target, flags, codes_out_ptr,
                                     alpha_out_ptr, scale_out_ptr, stream)


def accumulate_raw(codes_ptr: int, alpha_ptr: int, scale_ptr: int, grad_ptr: int, grad_dtype: int,
                   n: int, block: int, target: float, codes_out_ptr: int, alpha_out_ptr: int,
                   scale_out_ptr: int, stream: int = 0, flags: int = 0) -> int:
    return lib().tfp8_accumulate(codes_ptr, alpha_ptr, scale_ptr, grad_ptr, grad_dtype, n, block,
                                 target, flags, codes_out_ptr, alpha_out_ptr, scale_out_ptr, stream)


def compress_t_raw(x_ptr: int, x_dtype: int, rows: int, cols: int, ldx: int, offsets_ptr,
                   groups: int, block: int, target: float, codes_ptr: int, alpha_ptr: int,
                   scale_ptr: int, stream: int = 0, flags: int = 0) -> int:
    return lib().tfp8_compress_t(x_ptr, x_dtype, rows, cols, ldx, offsets_ptr, groups, block,
                                 target, flags, codes_ptr, alpha_ptr, scale_ptr, stream)


# An operand of a product is (codes_ptr, ld, alpha_ptr, scale_ptr, lds): row strides in codes and
# in scales.

def matmul_raw(a, b, m: int, n: int, k: int, block: int, out_ptr: int, out_dtype: int, ldc: int,
               stream: int = 0) -> int:
    return lib().tfp8_matmul(*a, *b, m, n, k, block, out_ptr, out_dtype, ldc, stream)


def matmul_grouped_raw(a, b, offsets_ptr: int, groups: int, m: int, n: int, k: int, block: int,
                       out_ptr: int, out_dtype: int, ldc: int, stream: int = 0) -> int:
    return lib().tfp8_matmul_grouped(*a, *b, offsets_ptr, groups, m, n, k, block, out_ptr,
                                     out_dtype, ldc, stream)


def matmul_grouped_t_raw(a, b, offsets_ptr: int, groups: int, rows: int, m: int, n: int,
                         block: int, out_ptr: int, out_dtype: int, stream: int = 0) -> int:
    return lib().tfp8_matmul_grouped_t(*a, *b, offsets_ptr, groups, rows, m, n, block, out_ptr,
                                       out_dtype, stream)


# The lists of tensors of the optimizer's calls are host memory: tables of tfp8_gradient and
# tfp8_adamw_tensor (include/tfp8.h), by address.

def grad_norm_raw(grads_ptr: int, count: int, block: int, max_norm: float, workspace_ptr: int,
                  workspace_bytes: int, norm_ptr: int, scale_ptr: int, stream: int = 0) -> int:
    return lib().tfp8_grad_norm(grads_ptr, count, block, max_norm, workspace_ptr, workspace_bytes,
                                norm_ptr, scale_ptr, stream)


def adamw_raw(tensors_ptr: int, count: int, block: int, bits: int, state, state_out, state_n: int,
              options, stream: int = 0) -> int:
    """state and state_out: the addresses (m, m_scale, v, v_scale)."""
    return lib().tfp8_adamw(tensors_ptr, count, block, bits, *state, *state_out, state_n, options,
                            stream)


def moe_layer_raw(x, router, up, down, tokens: int, experts: int, top_k: int, k: int, f: int,
                  block: int, flags: int, workspace_ptr: int, workspace_bytes: int, out,
                  stream: int = 0) -> int:
    """x and out are (address, dtype, row stride), router (address, dtype), up and down the addresses
    (codes, alpha, scale)."""
    return lib().tfp8_moe_layer(*x, *router, *up, *down, tokens, experts, top_k, k, f, block, flags,
                                workspace_ptr, workspace_bytes, *out, stream)


# ---------------------------------------------------------------------------- tensor wrappers

def _stream(t: torch.Tensor) -> int:
    # the raw handle of torch.cuda.current_stream(t.device), without making a Stream object
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _run(t: torch.Tensor, raw, *args):
    """raw(*args) with t's device as the current one, and its status checked."""
    if torch.cuda.current_device() == t.get_device():
        status = raw(*args)
    else:
        with torch.cuda.device(t.device):
            status = raw(*args)
    if status != 0:
        _check(status)


def _need_gpu(*ts):
    """Every tensor on the same GPU and contiguous (the library reads flat buffers)."""
    dev = None
    for t in ts:
        if not (isinstance(t, torch.Tensor) and t.is_cuda):
            raise ValueError("tfp8 operates on GPU tensors only (no CPU path)")
        if not t.is_contiguous():
            raise ValueError("tfp8 needs contiguous tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on different devices ({dev} and {t.device})")


def _need_buf(t: torch.Tensor, dtype: torch.dtype, numel: int, name: str):
    """A buffer the kernels read or write: its dtype and exact element count, checked here
    because the C ABI takes bare pointers and cannot."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")


def _blocks(n: int, block: int) -> int:
    if block not in SUPPORTED_BLOCKS:
        raise ValueError(f"block must be one of {SUPPORTED_BLOCKS}, got {block}")
    if n % block:
        raise ValueError(f"{n} elements are not a multiple of the block size {block}")
    return n // block


def compress(x: torch.Tensor, block: int = 128, target: float = 1.0, out=None, flags: int = 0):
    """x (bfloat16 or float32, any shape, numel % block == 0) ->
    (codes uint8 of x's shape, alpha float32 [numel/block], scale float32 [numel/block])."""
    _need_gpu(x)
    if x.dtype == torch.bfloat16:
        dt = BF16
    elif x.dtype == torch.float32:
        dt = F32
    else:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    n = x.numel()
    nb = _blocks(n, block)
    if out is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
        alpha = torch.empty(nb, dtype=torch.float32, device=x.device)
        scale = torch.empty(nb, dtype=torch.float32, device=x.device)
    else:
        codes, alpha, scale = out
        _need_gpu(x, codes, alpha, scale)
    _need_buf(codes, torch.uint8, n, "codes")
    _need_buf(alpha, torch.float32, nb, "alpha")
    _need_buf(scale, torch.float32, nb, "scale")
    _run(x, compress_raw, x.data_ptr(), dt, n, block, float(target), codes.data_ptr(),
         alpha.data_ptr(), scale.data_ptr(), _stream(x), flags)
    return codes, alpha, scale


def decompress(codes: torch.Tensor, alpha: torch.Tensor, scale: torch.Tensor, block: int = 128,
               dtype: torch.dtype = torch.float32, out=None, flags: int = 0):
    """Reconstruct a float32 or bfloat16 tensor of codes' shape."""
    _need_gpu(codes, alpha, scale)
    if dtype == torch.float32:
        dt = F32
    elif dtype == torch.bfloat16:
        dt = BF16
    else:
        raise ValueError(f"unsupported output dtype {dtype}")
    n = codes.numel()
    nb = _blocks(n, block)
    _need_buf(codes, torch.uint8, n, "codes")
    _need_buf(alpha, torch.float32, nb, "alpha")
    _need_buf(scale, torch.float32, nb, "scale")
    if out is None:
        out = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    else:
        _need_gpu(codes, out)
        _need_buf(out, dtype, n, "out")
    _run(codes, decompress_raw, codes.data_ptr(), alpha.data_ptr(), scale.data_ptr(), n, block,
         out.data_ptr(), dt, _stream(codes), flags)
    return out


def _peer_rows(t: torch.Tensor, dtype: torch.dtype, P: int, m: int, name: str) -> int:
    """A [P, m] view whose rows are contiguous, at any row stride (for example rows of one receive
    buffer); returns the row stride in elements."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError("tfp8 operates on GPU tensors only (no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or tuple(t.shape) != (P, m):
        raise ValueError(f"{name} must be [{P}, {m}], got {list(t.shape)}")
    if m > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if P > 1 else m


def reduce_fp8(codes: torch.Tensor, alpha: torch.Tensor, scale: torch.Tensor, block: int = 128,
               target: float = 1.0, out=None, flags: int = 0):
    """codes [P, ...], alpha and scale [P, nb] -> (codes [...], alpha [nb], scale [nb]).

    Contiguous stacks go to tfp8_reduce_fp8.  Otherwise codes must be a [P, n] view and alpha,
    scale [P, nb] views whose rows are contiguous but may lie at any stride, for example rows of
    one buffer holding a [codes | alpha | scale] message per peer; those go to
    tfp8_reduce_strided and give the same result."""
    if codes.dim() < 2:
        raise ValueError("codes must be stacked as [P, ...]")
    P = codes.shape[0]
    n = codes[0].numel()
    nb = _blocks(n, block)
    strided = not (codes.is_contiguous() and alpha.is_contiguous() and scale.is_contiguous())
    if strided:
        cst = _peer_rows(codes, torch.uint8, P, n, "codes")
        ast = _peer_rows(alpha, torch.float32, P, nb, "alpha")
        sst = _peer_rows(scale, torch.float32, P, nb, "scale")
        if not (codes.device == alpha.device == scale.device):
            raise ValueError("tensors on different devices")
    else:
        _need_gpu(codes, alpha, scale)
        _need_buf(codes, torch.uint8, P * n, "codes")
        _need_buf(alpha, torch.float32, P * nb, "alpha")
        _need_buf(scale, torch.float32, P * nb, "scale")
    if out is None:
        codes_out = torch.empty(codes.shape[1:], dtype=torch.uint8, device=codes.device)
        alpha_out = torch.empty(nb, dtype=torch.float32, device=codes.device)
        scale_out = torch.empty(nb, dtype=torch.float32, device=codes.device)
    else:
        codes_out, alpha_out, scale_out = out
        _need_gpu(codes_out, alpha_out, scale_out)
        if codes_out.device != codes.device:
            raise ValueError(
                f"tensors on different devices ({codes.device} and {codes_out.device})")
        _need_buf(codes_out, torch.uint8, n, "codes_out")
        _need_buf(alpha_out, torch.float32, nb, "alpha_out")
        _need_buf(scale_out, torch.float32, nb, "scale_out")
    if strided:
        _run(codes, reduce_strided_raw, codes.data_ptr(), cst, alpha.data_ptr(), ast,
             scale.data_ptr(), sst, P, n, block, float(target), codes_out.data_ptr(),
             alpha_out.data_ptr(), scale_out.data_ptr(), _stream(codes), flags)
    else:
        _run(codes, reduce_fp8_raw, codes.data_ptr(), alpha.data_ptr(), scale.data_ptr(), P, n,
             block, float(target), codes_out.data_ptr(), alpha_out.data_ptr(),
             scale_out.data_ptr(), _stream(codes), flags)
    return codes_out, alpha_out, scale_out


def accumulate(codes: torch.Tensor, alpha: torch.Tensor, scale: torch.Tensor, grad: torch.Tensor,
               block: int = 128, target: float = 1.0, out=None, flags: int = 0,
               inplace: bool = False):
    """Compressed main gradient + dense local gradient (bfloat16 or float32, same numel) ->
    compressed sum.  inplace=True overwrites (codes, alpha, scale) and returns them."""
    _need_gpu(codes, alpha, scale, grad)
    if grad.dtype == torch.bfloat16:
        dt = BF16
    elif grad.dtype == torch.float32:
        dt = F32
    else:
        raise ValueError(f"unsupported gradient dtype {grad.dtype}")
    n = codes.numel()
    if grad.numel() != n:
        raise ValueError("grad and codes must have the same number of elements")
    nb = _blocks(n, block)
    _need_buf(codes, torch.uint8, n, "codes")
    _need_buf(alpha, torch.float32, nb, "alpha")
    _need_buf(scale, torch.float32, nb, "scale")
    if inplace:
        if out is not None:
            raise ValueError("give either out or inplace=True, not both")
        out = (codes, alpha, scale)
    elif out is None:
        out = (torch.empty_like(codes), torch.empty_like(alpha), torch.empty_like(scale))
    else:
        _need_gpu(codes, *out)
        names = ("codes_out", "alpha_out", "scale_out")
        for t, ref, name in zip(out, (codes, alpha, scale), names):
            _need_buf(t, ref.dtype, ref.numel(), name)
    _run(codes, accumulate_raw, codes.data_ptr(), alpha.data_ptr(), scale.data_ptr(),
         grad.data_ptr(), dt, n, block, float(target), out[0].data_ptr(), out[1].data_ptr(),
         out[2].data_ptr(), _stream(codes), flags)
    return out


# ------------------------------------------------------------- products of compressed operands

def padded_rows(rows: int, groups: int = 1, block: int = 128) -> int:
    """Length of a compress_t row: room for `rows` rows in `groups` groups, each rounded up to a
    whole block, whatever the sizes of the groups."""
    if rows < 0 or not 1 <= groups <= MAX_GROUPS or block < 1:
        raise ValueError(f"padded_rows({rows}, {groups}, {block}): out of range")
    return (rows + groups * (block - 1)) // block * block


def _product_block(block: int):
    if block not in PRODUCT_BLOCKS:
        raise ValueError(f"block must be one of {PRODUCT_BLOCKS}, got {block}")


def _out_dtype(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return F32
    if dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"unsupported output dtype {dtype}")


def _offsets_of(offsets: torch.Tensor, t: torch.Tensor) -> int:
    """The number of groups that offsets cut, on t's device."""
    if not (isinstance(offsets, torch.Tensor) and offsets.is_cuda):
        raise ValueError("tfp8 operates on GPU tensors only (no CPU path)")
    if offsets.get_device() != t.get_device():
        raise ValueError(f"tensors on different devices ({t.device} and {offsets.device})")
    if offsets.dtype != torch.int64 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int64 vector")
    groups = offsets.numel() - 1
    if not 1 <= groups <= MAX_GROUPS:
        raise ValueError(f"offsets must have 2 to {MAX_GROUPS + 1} elements, got {groups + 1}")
    return groups


def _operand(t, block: int, dims: int, name: str):
    """(codes, alpha, scale) of an operand -> (shape of codes, its raw form).

    codes is uint8 [rows, k] (dims = 2, rows at any stride that is a multiple of 16) or contiguous
    [groups, rows, k]; alpha and scale are float32 with k / block values a row, [rows, k / block]
    with contiguous rows, or contiguous in any shape (as compress returns them)."""
    codes, alpha, scale = t
    # the common form, all contiguous; whatever fails here is looked at again below
    if (isinstance(codes, torch.Tensor) and isinstance(alpha, torch.Tensor)
            and isinstance(scale, torch.Tensor) and codes.dtype is torch.uint8
            and alpha.dtype is torch.float32 and scale.dtype is torch.float32
            and codes.is_contiguous() and alpha.is_contiguous() and scale.is_contiguous()
            and codes.get_device() == alpha.get_device() == scale.get_device() >= 0):
        shape = codes.shape
        if len(shape) == dims:
            k = shape[-1]
            if k % block == 0 and alpha.numel() == scale.numel() == codes.numel() // block:
                return shape, (codes.data_ptr(), k, alpha.data_ptr(), scale.data_ptr(), k // block)
    for x, dt, what in ((codes, torch.uint8, "codes"), (alpha, torch.float32, "alpha"),
                        (scale, torch.float32, "scale")):
        if not (isinstance(x, torch.Tensor) and x.is_cuda):
            raise ValueError("tfp8 operates on GPU tensors only (no CPU path)")
        if x.dtype != dt:
            raise ValueError(f"{what} of {name} must be {dt}, got {x.dtype}")
        if x.device != codes.device:
            raise ValueError(f"tensors on different devices ({codes.device} and {x.device})")
    if codes.dim() != dims:
        raise ValueError(f"codes of {name} must have {dims} dimensions, got {list(codes.shape)}")
    rows, k = codes.shape[-2], codes.shape[-1]
    if k % block:
        raise ValueError(f"rows of {name} have {k} elements, not a multiple of the block size "
                         f"{block}")
    nb = k // block
    ld = k
    if not codes.is_contiguous():
        if dims != 2 or (k > 1 and codes.stride(1) != 1):
            raise ValueError(f"codes of {name} must have contiguous rows")
        ld = codes.stride(0) if rows > 1 else k
    strides = []
    for x, what in ((alpha, "alpha"), (scale, "scale")):
        if x.numel() != codes.numel() // block:
            raise ValueError(f"{what} of {name} must have {codes.numel() // block} elements, got "
                             f"{x.numel()}")
        if x.is_contiguous():
            strides.append(nb)
        elif dims == 2 and tuple(x.shape) == (rows, nb) and (nb <= 1 or x.stride(1) == 1):
            strides.append(x.stride(0) if rows > 1 else nb)
        else:
            raise ValueError(f"{what} of {name} must be [{rows}, {nb}] with contiguous rows")
    if strides[0] != strides[1]:
        raise ValueError(f"alpha and scale of {name} must have the same row stride")
    return codes.shape, (codes.data_ptr(), ld, alpha.data_ptr(), scale.data_ptr(), strides[0])


def _product_out(out, shape, dtype: torch.dtype, a, b):
    """(the output, its row stride) of a product of a and b, whose devices are compared: a new
    tensor, or `out` checked, whose rows must be contiguous."""
    if a[0].get_device() != b[0].get_device():
        raise ValueError(f"tensors on different devices ({a[0].device} and {b[0].device})")
    device = a[0].device
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device), shape[-1]
    if not (isinstance(out, torch.Tensor) and out.is_cuda):
        raise ValueError("tfp8 operates on GPU tensors only (no CPU path)")
    if out.device != device:
        raise ValueError(f"tensors on different devices ({device} and {out.device})")
    if out.dtype != dtype or tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must be {dtype} {list(shape)}, got {out.dtype} {list(out.shape)}")
    if out.numel() and shape[-1] > 1 and out.stride(-1) != 1:
        raise ValueError("the rows of out must be contiguous")
    return out, out.stride(-2) if shape[-2] > 1 else shape[-1]


def compress_t(x: torch.Tensor, block: int = 128, target: float = 1.0, offsets=None, out=None,
               flags: int = 0):
    """Compress x^T: x [rows, cols] (bfloat16 or float32, rows at any stride) -> the operand
    (codes uint8 [cols, kp], alpha, scale float32 [cols, kp / block]) whose blocks run along the
    rows of x, for products that contract over them.

    offsets (int64 [groups + 1] on the GPU, ascending) cuts the rows into groups, [offsets[g],
    offsets[g + 1]); each group starts at a multiple of the block in the output, kp =
    padded_rows(rows, groups, block), what no row fills counts as zeros, and rows before offsets[0]
    or past offsets[-1] are left out.  flags: 0 or FLAG_NO_ROTATION."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        raise ValueError("tfp8 operates on GPU tensors only (no CPU path)")
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, cols], got {list(x.shape)}")
    if x.dtype == torch.bfloat16:
        dt = BF16
    elif x.dtype == torch.float32:
        dt = F32
    else:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    _product_block(block)
    rows, cols = x.shape
    if rows and cols > 1 and x.stride(1) != 1:
        raise ValueError("the rows of x must be contiguous")
    ldx = x.stride(0) if rows > 1 else cols
    groups = 1 if offsets is None else _offsets_of(offsets, x)
    kp = padded_rows(rows, groups, block)
    if out is None:
        out = (torch.empty((cols, kp), dtype=torch.uint8, device=x.device),
               torch.empty((cols, kp // block), dtype=torch.float32, device=x.device),
               torch.empty((cols, kp // block), dtype=torch.float32, device=x.device))
        codes, alpha, scale = out
    else:
        codes, alpha, scale = out
        _need_gpu(codes, alpha, scale)
        if codes.device != x.device:
            raise ValueError(f"tensors on different devices ({x.device} and {codes.device})")
        _need_buf(codes, torch.uint8, cols * kp, "codes")
        _need_buf(alpha, torch.float32, cols * (kp // block), "alpha")
        _need_buf(scale, torch.float32, cols * (kp // block), "scale")
    _run(x, compress_t_raw, x.data_ptr(), dt, rows, cols, ldx,
         None if offsets is None else offsets.data_ptr(), groups, block, float(target),
         codes.data_ptr(), alpha.data_ptr(), scale.data_ptr(), _stream(x), flags)
    return codes, alpha, scale


def matmul(a, b, block: int = 128, dtype: torch.dtype = torch.bfloat16, out=None):
    """A^ B^T of two compressed operands a = (codes [m, k], alpha, scale) and b = (codes [n, k],
    alpha, scale), compressed in blocks along k with the same rotation -> [m, n] float32 or
    bfloat16.

    float32 outputs sum in float32 throughout.  bfloat16 outputs come from the 8-bit matrix
    instructions, at twice the rate: they add eight neighbouring products with 14 bits from the largest
    one's down, about 1.4e-5 of the result, which bfloat16's rounding covers unless larger terms
    cancel.  The grouped products do the same."""
    _product_block(block)
    dt = _out_dtype(dtype)
    (m, k), ra = _operand(a, block, 2, "a")
    (n, kb), rb = _operand(b, block, 2, "b")
    if k != kb:
        raise ValueError(f"a and b have rows of {k} and {kb} elements")
    out, ldc = _product_out(out, (m, n), dtype, a, b)
    _run(out, matmul_raw, ra, rb, m, n, k, block, out.data_ptr(), dt, ldc, _stream(out))
    return out


def matmul_grouped(a, b, offsets: torch.Tensor, block: int = 128,
                   dtype: torch.dtype = torch.bfloat16, out=None):
    """Rows grouped by expert: a = (codes [m, k], ...) with the rows of group g at
    [offsets[g], offsets[g + 1]), b = (codes [groups, n, k], ...) -> [m, n], each row times its
    group's b.  Rows before offsets[0] and past offsets[-1] become zeros."""
    _product_block(block)
    dt = _out_dtype(dtype)
    (m, k), ra = _operand(a, block, 2, "a")
    (g, n, kb), rb = _operand(b, block, 3, "b")
    if k != kb:
        raise ValueError(f"a and b have rows of {k} and {kb} elements")
    groups = _offsets_of(offsets, a[0])
    if groups != g:
        raise ValueError(f"offsets cut {groups} groups and b holds {g}")
    out, ldc = _product_out(out, (m, n), dtype, a, b)
    _run(out, matmul_grouped_raw, ra, rb, offsets.data_ptr(), groups, m, n, k, block,
         out.data_ptr(), dt, ldc, _stream(out))
    return out


def matmul_grouped_t(a, b, offsets: torch.Tensor, rows: int, block: int = 128,
                     dtype: torch.dtype = torch.float32, out=None):
    """Grouped along the contraction: a and b are compress_t's, with the same offsets, of matrices
    [rows, m] and [rows, n] -> [groups, m, n], for each group the product over its own rows (with
    a of dY and b of X: each expert's weight gradient).  Zeros for an empty group."""
    _product_block(block)
    dt = _out_dtype(dtype)
    (m, k), ra = _operand(a, block, 2, "a")
    (n, kb), rb = _operand(b, block, 2, "b")
    groups = _offsets_of(offsets, a[0])
    kp = padded_rows(rows, groups, block)
    if k != kp or kb != kp:
        raise ValueError(f"{rows} rows in {groups} groups are {kp} elements a row, got {k} and {kb}")
    out, _ = _product_out(out, (groups, m, n), dtype, a, b)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    _run(out, matmul_grouped_t_raw, ra, rb, offsets.data_ptr(), groups, rows, m, n, block,
         out.data_ptr(), dt, _stream(out))
    return out


def moe_layer(x: torch.Tensor, router: torch.Tensor, up, down, top_k: int, block: int = 128,
              renormalize: bool = True, dtype: torch.dtype = torch.bfloat16, flags: int = 0,
              out=None):
    """A whole layer of gated experts for up to MOE_TOKENS tokens, read from the experts' codes:

      logits = x router^T, the top_k largest of each token (the lower index first among equals),
      w = softmax of the chosen logits (renormalize=False: the chosen ones' part of the softmax of all),
      y[t] = sum over the chosen e of w[t, e] W2_e (silu(W1_e x[t]) * (W3_e x[t])).

    x [tokens, k] and router [experts, k]: bfloat16 or float32; up = (codes [experts, 2 f, k], alpha,
    scale), the rows of W1 before those of W3, compressed along k; down = (codes [experts, k, f], alpha,
    scale), compressed along f.  -> [tokens, k], bfloat16 or float32 (dtype).  flags: 0 or
    FLAG_NO_ROTATION, as the weights were compressed.  It records no graph, and refuses inputs that want
    a gradient while gradients are on.  More tokens: sort them by expert and use matmul_grouped, whose
    products run on compressed activations."""
    _product_block(block)
    dt = _out_dtype(dtype)
    if flags & ~FLAG_NO_ROTATION:
        _check(-6)  # TFP8_E_ARG, as the C call gives it for the flags that it does not know
    for t, name in ((x, "x"), (router, "router")):
        if not (isinstance(t, torch.Tensor) and t.is_cuda):
            raise ValueError("tfp8 operates on GPU tensors only (no CPU path)")
        if t.dim() != 2:
            raise ValueError(f"{name} must have 2 dimensions, got {list(t.shape)}")
        if t.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"unsupported {name} dtype {t.dtype}")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient, which moe_layer does not pass back")
    tokens, k = x.shape
    (experts, f2, ku), ru = _operand(up, block, 3, "up")
    (ed, kd, f), rd = _operand(down, block, 3, "down")
    if router.shape[0] != experts or ed != experts:
        raise ValueError(f"{router.shape[0]} rows of router, {experts} experts in up and {ed} in down")
    if not (router.shape[1] == ku == kd == k) or f2 != 2 * f:
        raise ValueError(f"x is [.., {k}], router [.., {router.shape[1]}], up [.., {f2}, {ku}] and "
                         f"down [.., {kd}, {f}]")
    if tokens > MOE_TOKENS or experts > MOE_EXPERTS:
        raise ValueError(f"at most {MOE_TOKENS} tokens and {MOE_EXPERTS} experts, got {tokens} and "
                         f"{experts}")
    if not 1 <= top_k <= experts:
        raise ValueError(f"top_k must be 1 to {experts}, got {top_k}")
    for t, name in ((router, "router"), (up[0], "up"), (down[0], "down")):
        if t.get_device() != x.get_device():
            raise ValueError(f"{name} and x on different devices ({t.device} and {x.device})")
    if not router.is_contiguous() or (tokens and x.stride(1) != 1):
        raise ValueError("router and the rows of x must be contiguous")
    given = out is not None
    out, ldo = _product_out(out, (tokens, k), dtype, (x,), up)
    nbytes = lib().tfp8_moe_workspace(tokens, experts, top_k, k, f)
    workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    raw = lambda t: (t.data_ptr(), BF16 if t.dtype == torch.bfloat16 else F32)
    _run(x, moe_layer_raw, (*raw(x), x.stride(0) if tokens > 1 else k), raw(router),
         (ru[0], ru[2], ru[3]), (rd[0], rd[2], rd[3]), tokens, experts, top_k, k, f, block,
         flags | (0 if renormalize else _MOE_ALL_EXPERTS), workspace.data_ptr(), nbytes,
         (out.data_ptr(), dt, ldo), _stream(x))
    if given:  # a graph that has saved it is not to be run backward through its new values
        torch.autograd.graph.increment_version(out)
    return out


from .optimizer import adamw, adamw_state, grad_norm  # noqa: E402  (it takes the helpers above)
