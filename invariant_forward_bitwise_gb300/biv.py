"""Python binding of libbiv: the C-ABI entry points of ``include/biv.h`` under
the same names, taking torch CUDA tensors.  Argument marshalling only: every
step runs in the library's CUDA kernels.  There is no CPU fallback; a missing
or unloadable library raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from typing import Dict, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbiv.so")

BIV_OK, BIV_ERR_INVALID, BIV_ERR_UNSUPPORTED, BIV_ERR_WORKSPACE, BIV_ERR_CUDA, BIV_ERR_TIMEOUT = range(6)
MODE_INVARIANT, MODE_FAST = 0, 1
BF16, F32, E4M3 = 0, 1, 2
LOSS_TOKEN_MEAN, LOSS_SEQ_MEAN, LOSS_SUM = 0, 1, 2
ROUND_NEAREST, ROUND_STOCHASTIC = 0, 1

EXPORTS = [
    "biv_version", "biv_last_error", "biv_device_sm_count", "biv_poll_error",
    "biv_selftest_timeout", "biv_embed", "biv_add_rmsnorm", "biv_add_rmsnorm_partials", "biv_silu_mul",
    "biv_rope_table", "biv_qk_norm_rope", "biv_kv_store_bf16", "biv_kv_fp8_quant", "biv_qkv_finalize", "biv_silu_mul_partials",
    "biv_kv_fp8_gather", "biv_attention_workspace", "biv_attention", "biv_attention_noalloc",
    "biv_gemm_workspace", "biv_gemm_partials", "biv_gemm",
    "biv_act_quant_fp8", "biv_silu_mul_quant_fp8", "biv_topk", "biv_router_topk", "biv_moe_dispatch", "biv_gather_rows",
    "biv_moe_combine", "biv_logprob", "biv_lm_head_logprob_workspace", "biv_lm_head_logprob",
    "biv_ssd_workspace", "biv_ssd_scan",
    "biv_causal_conv1d", "biv_gated_rmsnorm", "biv_nvfp4_dequant",
    "biv_gemm_nvfp4_workspace", "biv_gemm_nvfp4",
    "biv_rmsnorm_backward", "biv_silu_mul_backward", "biv_logprob_backward", "biv_attention_backward",
    "biv_policy_loss_workspace", "biv_policy_loss", "biv_policy_loss_logits",
    "biv_lm_head_loss_workspace", "biv_lm_head_loss",
    "biv_lm_head_backward_workspace", "biv_lm_head_backward",
    "biv_add_rmsnorm_fp8", "biv_rmsnorm_backward_fp8_workspace", "biv_rmsnorm_backward_fp8",
    "biv_silu_mul_keep_fp8", "biv_silu_mul_backward_fp8",
    "biv_opt_plan", "biv_grad_norm_workspace", "biv_grad_norm", "biv_adamw",
]


class BivError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libbiv status {status}: {msg}")
        self.status = status


class GemmDesc(C.Structure):
    _fields_ = [("M", C.c_int), ("N", C.c_int), ("K", C.c_int),
                ("a_dtype", C.c_int), ("b_dtype", C.c_int), ("c_dtype", C.c_int),
                ("A", C.c_void_p), ("lda", C.c_int64),
                ("B", C.c_void_p), ("ldb", C.c_int64),
                ("C", C.c_void_p), ("ldc", C.c_int64),
                ("sa", C.c_void_p), ("ld_sa", C.c_int64),
                ("sb", C.c_void_p),
                ("group_offsets", C.c_void_p), ("groups", C.c_int),
                ("mode", C.c_int), ("defer_fold", C.c_int), ("b_early", C.c_int)]


class Partials(C.Structure):
    """Chunk partials a GEMM left for its consumer (see include/biv.h)."""
    _fields_ = [("p", C.c_void_p), ("chunks", C.c_int), ("ld", C.c_int64),
                ("chunk_stride", C.c_int64)]


class AttnDesc(C.Structure):
    _fields_ = [("q", C.c_void_p), ("q_stride", C.c_int64),
                ("out", C.c_void_p), ("out_stride", C.c_int64),
                ("T", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int),
                ("row_seq", C.c_void_p), ("row_pos", C.c_void_p),
                ("qblocks", C.c_void_p), ("nqblocks", C.c_int),
                ("max_rows_per_block", C.c_int),
                ("kv_dtype", C.c_int),
                ("k_cache", C.c_void_p), ("v_cache", C.c_void_p),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("block_table", C.c_void_p), ("max_pages", C.c_int),
                ("page", C.c_int), ("kv_split", C.c_int), ("max_ctx", C.c_int),
                ("topk_idx", C.c_void_p), ("topk_stride", C.c_int64), ("topk", C.c_int),
                ("scale", C.c_float), ("mode", C.c_int), ("num_pages", C.c_int)]


class SSDDesc(C.Structure):
    _fields_ = [("x", C.c_void_p), ("x_stride", C.c_int64),
                ("dt", C.c_void_p), ("dt_stride", C.c_int64),
                ("A", C.c_void_p),
                ("B", C.c_void_p), ("B_stride", C.c_int64),
                ("C", C.c_void_p), ("C_stride", C.c_int64),
                ("D", C.c_void_p),
                ("y", C.c_void_p), ("y_stride", C.c_int64),
                ("H", C.c_int), ("P", C.c_int), ("N", C.c_int), ("chunk", C.c_int),
                ("nseq", C.c_int),
                ("row0", C.c_void_p), ("n", C.c_void_p), ("pos0", C.c_void_p),
                ("max_n", C.c_int),
                ("state", C.c_void_p), ("buf_x", C.c_void_p), ("buf_B", C.c_void_p),
                ("buf_C", C.c_void_p), ("buf_dt", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class ConvDesc(C.Structure):
    _fields_ = [("u", C.c_void_p), ("u_stride", C.c_int64),
                ("col_x", C.c_int), ("col_dt", C.c_int), ("channels", C.c_int), ("heads", C.c_int),
                ("width", C.c_int),
                ("conv_w", C.c_void_p), ("conv_b", C.c_void_p), ("dt_bias", C.c_void_p),
                ("out", C.c_void_p), ("out_stride", C.c_int64),
                ("dt_out", C.c_void_p), ("dt_stride", C.c_int64),
                ("T", C.c_int),
                ("row_seq", C.c_void_p), ("row_pos", C.c_void_p),
                ("nseq", C.c_int),
                ("row0", C.c_void_p), ("n", C.c_void_p), ("pos0", C.c_void_p),
                ("state", C.c_void_p)]


class AttnBwdDesc(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("dout", C.c_void_p),
                ("dq", C.c_void_p), ("dk", C.c_void_p), ("dv", C.c_void_p),
                ("Tq", C.c_int), ("Tk", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int),
                ("q_pos", C.c_void_p), ("k_pos", C.c_void_p), ("scale", C.c_float),
                ("workspace", C.c_void_p)]


class PolicyDesc(C.Structure):
    _fields_ = [("T", C.c_int), ("nseq", C.c_int),
                ("seq_start", C.c_void_p), ("mask", C.c_void_p),
                ("old_lp", C.c_void_p), ("ref_lp", C.c_void_p),
                ("adv", C.c_void_p), ("adv_per_row", C.c_int),
                ("clip_lo", C.c_float), ("clip_hi", C.c_float), ("dual_clip", C.c_float),
                ("kl_coef", C.c_float), ("ent_coef", C.c_float),
                ("reduce", C.c_int), ("norm", C.c_float),
                ("stats", C.c_void_p), ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class LmLossDesc(C.Structure):
    _fields_ = [("T", C.c_int), ("V", C.c_int), ("K", C.c_int),
                ("h", C.c_void_p), ("ldh", C.c_int64), ("W", C.c_void_p), ("ldw", C.c_int64),
                ("target", C.c_void_p), ("weight", C.c_void_p), ("ignore_index", C.c_int),
                ("z_coef", C.c_float), ("reduce", C.c_int), ("norm", C.c_float),
                ("lp", C.c_void_p), ("lse", C.c_void_p), ("dlp", C.c_void_p), ("dlse", C.c_void_p),
                ("stats", C.c_void_p), ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class LmGradDesc(C.Structure):
    _fields_ = [("T", C.c_int), ("V", C.c_int), ("K", C.c_int),
                ("h", C.c_void_p), ("ldh", C.c_int64), ("W", C.c_void_p), ("ldw", C.c_int64),
                ("target", C.c_void_p), ("lse", C.c_void_p), ("dlp", C.c_void_p), ("dlse", C.c_void_p),
                ("dh", C.c_void_p), ("lddh", C.c_int64), ("dh_dtype", C.c_int),
                ("dW", C.c_void_p), ("lddw", C.c_int64), ("dw_dtype", C.c_int),
                ("accumulate", C.c_int), ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


class NormFp8Desc(C.Structure):
    _fields_ = [("x", C.c_void_p), ("x_stride", C.c_int64),
                ("residual", C.c_void_p), ("r_stride", C.c_int64),
                ("residual_out", C.c_void_p), ("ro_stride", C.c_int64),
                ("w", C.c_void_p), ("y", C.c_void_p), ("y_stride", C.c_int64),
                ("codes", C.c_void_p), ("scales", C.c_void_p),
                ("keep", C.c_void_p), ("keep_scales", C.c_void_p), ("inv", C.c_void_p),
                ("rows", C.c_int), ("d", C.c_int), ("eps", C.c_float)]


class NormBwdFp8Desc(C.Structure):
    _fields_ = [("keep", C.c_void_p), ("keep_scales", C.c_void_p), ("inv", C.c_void_p), ("w", C.c_void_p),
                ("dy", C.c_void_p), ("dy_stride", C.c_int64), ("dy_dtype", C.c_int),
                ("dres", C.c_void_p), ("dres_stride", C.c_int64),
                ("dx", C.c_void_p), ("dx_stride", C.c_int64), ("dx_dtype", C.c_int),
                ("dw", C.c_void_p), ("accumulate", C.c_int), ("rows", C.c_int), ("d", C.c_int),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


_FORMATS = {C.c_void_p: "P", C.c_int: "i", C.c_int64: "q", C.c_float: "f", C.c_size_t: "N"}


def _packer(desc):
    """Packs the values of a descriptor (0 for no pointer) in a quarter of the time
    that ctypes takes to make one."""
    f = "".join(_FORMATS[kind] for _, kind in desc._fields_)
    s = struct.Struct(f"{f}{C.sizeof(desc) - struct.calcsize(f)}x")
    return s.pack


_pack_loss, _pack_grad = _packer(LmLossDesc), _packer(LmGradDesc)
_pack_norm, _pack_norm_bwd = _packer(NormFp8Desc), _packer(NormBwdFp8Desc)


class OptTensor(C.Structure):
    _fields_ = [("param", C.c_void_p), ("master", C.c_void_p), ("grad", C.c_void_p),
                ("m", C.c_void_p), ("v", C.c_void_p),
                ("m_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("numel", C.c_int64), ("first_chunk", C.c_int64), ("rng_base", C.c_int64),
                ("lr_scale", C.c_float), ("weight_decay", C.c_float),
                ("param_dtype", C.c_int32), ("grad_dtype", C.c_int32), ("state_dtype", C.c_int32),
                ("vec", C.c_int32)]


class AdamWDesc(C.Structure):
    _fields_ = [("tensors", C.c_void_p), ("n", C.c_int), ("kinds", C.c_int), ("chunks", C.c_int64),
                ("lr", C.c_void_p), ("clip", C.c_void_p), ("step", C.c_void_p),
                ("beta1", C.c_double), ("beta2", C.c_double), ("eps", C.c_float),
                ("rounding", C.c_int), ("seed", C.c_uint64)]


_lib: Optional[C.CDLL] = None


def load(path: str = LIB_PATH) -> C.CDLL:
    """Load libbiv.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libbiv.so not found at {path}: run invariant_forward_bitwise_gb300.build.build()")
    lib = C.CDLL(path)
    P, I, I64, F, D_ = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_double
    sig = {
        "biv_version": ([], I), "biv_last_error": ([], C.c_char_p),
        "biv_device_sm_count": ([], I), "biv_poll_error": ([P, P], I),
        "biv_selftest_timeout": ([C.c_uint64, P], I),
        "biv_embed": ([P, P, I, I, I, P, I64, P], I),
        "biv_add_rmsnorm": ([P, I64, P, I64, P, P, I64, I, I, F, P], I),
        "biv_add_rmsnorm_partials": ([P, P, I64, P, P, I64, I, I, F, P], I),
        "biv_qkv_finalize": ([P, I64, P, I, I, I, I, P, P, P, I, P, F, P, I, P, P, P, P, P], I),
        "biv_gemm_partials": ([P, P, P], I),
        "biv_silu_mul": ([P, I64, P, I64, I, I, P], I),
        "biv_silu_mul_partials": ([P, P, I64, I, I, P], I),
        "biv_rope_table": ([D_, I, I, P, P], I),
        "biv_qk_norm_rope": ([P, I64, I, I, I, I, P, P, P, I, P, F, P], I),
        "biv_kv_store_bf16": ([P, P, I64, P, I, I, I, P, P, P], I),
        "biv_kv_fp8_quant": ([P, P, I64, P, I, I, I, P, P, P, P, P], I),
        "biv_kv_fp8_gather": ([P, P, P, I, P, P, I, I, I, I, P, P], I),
        "biv_attention_workspace": ([P, P], I), "biv_attention": ([P, P, C.c_size_t, P], I),
        "biv_attention_noalloc": ([P, P], I),
        "biv_gemm_workspace": ([P, P], I), "biv_gemm": ([P, P, C.c_size_t, P], I),
        "biv_act_quant_fp8": ([P, I64, I, I, P, P, P], I),
        "biv_silu_mul_quant_fp8": ([P, I64, I, I, P, P, P], I),
        "biv_topk": ([P, I64, P, I, I, I, P, P], I),
        "biv_router_topk": ([P, I64, I, I, I, P, P, P], I),
        "biv_moe_dispatch": ([P, I, I, I, P, P, P, P], I),
        "biv_gather_rows": ([P, I64, P, I, I, I, P, I64, P], I),
        "biv_moe_combine": ([P, P, P, P, P, I, I, I, P], I),
        "biv_logprob": ([P, I64, P, I, I, P, P], I),
        "biv_lm_head_logprob_workspace": ([I, I, P], I),
        "biv_lm_head_logprob": ([P, I64, P, I64, I, I, I, P, I, P, P, C.c_size_t, P], I),
        "biv_ssd_workspace": ([P, P], I), "biv_ssd_scan": ([P, P], I),
        "biv_causal_conv1d": ([P, P], I),
        "biv_gated_rmsnorm": ([P, I64, P, I64, P, P, I64, I, I, F, P], I),
        "biv_nvfp4_dequant": ([P, P, I, I, P, P], I),
        "biv_gemm_nvfp4_workspace": ([I, I, I, I, I, P], I),
        "biv_gemm_nvfp4": ([P, I64, P, P, I, I, I, P, I64, I, I, P, C.c_size_t, P], I),
        "biv_rmsnorm_backward": ([P, I64, P, P, I64, P, I64, P, I, I, F, P, C.c_size_t, P], I),
        "biv_silu_mul_backward": ([P, I64, P, I64, P, I64, I, I, P], I),
        "biv_logprob_backward": ([P, I64, P, P, I, I, P, I64, P], I),
        "biv_attention_backward": ([P, P], I),
        "biv_policy_loss_workspace": ([I, I, P], I), "biv_policy_loss": ([P, P, P, P], I),
        "biv_policy_loss_logits": ([P, P, I64, I, P, I, F, P, P, P, I64, I, P], I),
        "biv_lm_head_loss_workspace": ([I, I, P], I), "biv_lm_head_loss": ([P, P], I),
        "biv_lm_head_backward_workspace": ([I, I, I, I, I, P], I), "biv_lm_head_backward": ([P, P], I),
        "biv_add_rmsnorm_fp8": ([P, P], I),
        "biv_rmsnorm_backward_fp8_workspace": ([I, I, P], I), "biv_rmsnorm_backward_fp8": ([P, P], I),
        "biv_silu_mul_keep_fp8": ([P, I64, P, I64, P, P, I, I, P], I),
        "biv_silu_mul_backward_fp8": ([P, P, P, I64, I, P, I64, I, P, I64, I, I, P], I),
        "biv_opt_plan": ([P, I, P, P], I), "biv_grad_norm_workspace": ([I64, P], I),
        "biv_grad_norm": ([P, I, I64, F, P, P, C.c_size_t, P], I), "biv_adamw": ([P, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name, None)
        if fn is None:
            continue
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def missing_exports(path: str = LIB_PATH) -> list:
    lib = C.CDLL(path)
    return [n for n in EXPORTS if not hasattr(lib, n)]


# ------------------------------------------------------------- helpers ----
def _p(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


# the current stream's handle without a Stream object around it, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# the current device, without the checks of torch.cuda.current_device()
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_device())
    return torch.cuda.current_stream().cuda_stream


def _check(st: int, what: str):
    if st != BIV_OK:
        raise BivError(st, f"{what}: {load().biv_last_error().decode()}")


def _rs(t: torch.Tensor) -> int:
    """row stride (elements) of a 2-D view."""
    return t.stride(0) if t.dim() >= 2 else t.shape[-1]


def _bf16_ok(*ts):
    for t in ts:
        if t is not None:
            assert t.is_cuda and t.dtype == torch.bfloat16, "expected a CUDA bf16 tensor"


# ------------------------------------------------------------ entry points --
def biv_version() -> int:
    return load().biv_version()


def biv_device_sm_count() -> int:
    return load().biv_device_sm_count()


def biv_poll_error(stream=None) -> int:
    code = C.c_int(0)
    st = load().biv_poll_error(_stream(stream), C.byref(code))
    if st not in (BIV_OK, BIV_ERR_TIMEOUT, BIV_ERR_INVALID):
        _check(st, "biv_poll_error")
    return code.value


def biv_selftest_timeout(limit_ns: int, stream=None):
    _check(load().biv_selftest_timeout(int(limit_ns), _stream(stream)), "biv_selftest_timeout")


def biv_embed(ids, table, h, stream=None):
    _bf16_ok(table, h)
    _check(load().biv_embed(_p(ids), _p(table), table.shape[0], ids.shape[0], table.shape[1],
                            _p(h), _rs(h), _stream(stream)), "biv_embed")


def biv_add_rmsnorm(x, residual, w, y, eps, stream=None):
    """residual may be None; rows = x.shape[0]."""
    _bf16_ok(x, residual, w, y)
    rows, d = x.shape[0], x.shape[-1]
    _check(load().biv_add_rmsnorm(_p(x), _rs(x), _p(residual), _rs(residual) if residual is not None else 0,
                                  _p(w), _p(y), _rs(y), rows, d, float(eps), _stream(stream)),
           "biv_add_rmsnorm")


def biv_silu_mul(gate_up, y, stream=None):
    _bf16_ok(gate_up, y)
    _check(load().biv_silu_mul(_p(gate_up), _rs(gate_up), _p(y), _rs(y), gate_up.shape[0],
                               y.shape[-1], _stream(stream)), "biv_silu_mul")


def biv_rope_table(theta, D, max_pos, out, stream=None):
    assert out.dtype == torch.float32 and out.numel() >= 2 * max_pos * (D // 2)
    _check(load().biv_rope_table(float(theta), D, max_pos, _p(out), _stream(stream)), "biv_rope_table")


def biv_add_rmsnorm_partials(xp: "Partials", residual, w, y, rows, eps, stream=None):
    """x given as GEMM chunk partials; rows/d from the arguments."""
    _bf16_ok(residual, w, y)
    d = y.shape[-1]
    _check(load().biv_add_rmsnorm_partials(C.byref(xp), _p(residual),
                                           _rs(residual) if residual is not None else 0, _p(w), _p(y),
                                           _rs(y), rows, d, float(eps), _stream(stream)),
           "biv_add_rmsnorm_partials")


def biv_silu_mul_partials(gp: "Partials", y, rows, stream=None):
    """gate_up given as GEMM chunk partials; I = y.shape[-1]."""
    _bf16_ok(y)
    _check(load().biv_silu_mul_partials(C.byref(gp), _p(y), _rs(y), rows, y.shape[-1],
                                        _stream(stream)), "biv_silu_mul_partials")


def biv_qkv_finalize(qkv, T, Hq, Hkv, D, q_w, k_w, cos_sin, max_pos, pos, eps, slot, kv_dtype,
                     k_cache, v_cache, k_scale=None, v_scale=None, partials: Optional["Partials"] = None,
                     stream=None):
    _check(load().biv_qkv_finalize(_p(qkv), _rs(qkv), C.byref(partials) if partials is not None else None,
                                   T, Hq, Hkv, D, _p(q_w), _p(k_w), _p(cos_sin), max_pos, _p(pos),
                                   float(eps), _p(slot), kv_dtype, _p(k_cache), _p(v_cache), _p(k_scale),
                                   _p(v_scale), _stream(stream)), "biv_qkv_finalize")


def biv_gemm_partials(desc: GemmDesc, ws: Optional[torch.Tensor]) -> "Partials":
    out = Partials()
    _check(load().biv_gemm_partials(C.byref(desc), _p(ws), C.byref(out)), "biv_gemm_partials")
    return out


def biv_qk_norm_rope(qkv, T, Hq, Hkv, D, q_w, k_w, cos_sin, max_pos, pos, eps, stream=None):
    _check(load().biv_qk_norm_rope(_p(qkv), _rs(qkv), T, Hq, Hkv, D, _p(q_w), _p(k_w), _p(cos_sin),
                                   max_pos, _p(pos), float(eps), _stream(stream)), "biv_qk_norm_rope")


def biv_kv_store_bf16(k, v, row_stride, slot, T, Hkv, D, k_cache, v_cache, stream=None):
    _check(load().biv_kv_store_bf16(_p(k), _p(v), row_stride, _p(slot), T, Hkv, D, _p(k_cache),
                                    _p(v_cache), _stream(stream)), "biv_kv_store_bf16")


def biv_kv_fp8_quant(k, v, row_stride, slot, T, Hkv, D, kc, vc, ks, vs, stream=None):
    _check(load().biv_kv_fp8_quant(_p(k), _p(v), row_stride, _p(slot), T, Hkv, D, _p(kc), _p(vc),
                                   _p(ks), _p(vs), _stream(stream)), "biv_kv_fp8_quant")


def biv_kv_fp8_gather(codes, scales, block_table, ctx_len, out_row0, Hkv, D, page, out, stream=None):
    _check(load().biv_kv_fp8_gather(_p(codes), _p(scales), _p(block_table), block_table.shape[1],
                                    _p(ctx_len), _p(out_row0), ctx_len.shape[0], Hkv, D, page,
                                    _p(out), _stream(stream)), "biv_kv_fp8_gather")


def biv_attention_workspace(desc: AttnDesc) -> int:
    n = C.c_size_t(0)
    _check(load().biv_attention_workspace(C.byref(desc), C.byref(n)), "biv_attention_workspace")
    return n.value


def biv_attention(desc: AttnDesc, ws: Optional[torch.Tensor], stream=None):
    _check(load().biv_attention(C.byref(desc), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                _stream(stream)), "biv_attention")


def biv_attention_noalloc(desc: AttnDesc, stream=None):
    """biv_attention without a caller workspace (see include/biv.h)."""
    _check(load().biv_attention_noalloc(C.byref(desc), _stream(stream)), "biv_attention_noalloc")


def gemm_desc(A, B, Cout, mode=MODE_INVARIANT, sa=None, sb=None, group_offsets=None, groups=0,
              M=None, b_early=False) -> GemmDesc:
    """b_early: B is loaded while the calls ahead may still run (see
    include/biv.h); not for a B that the call just before writes."""
    dt = {torch.bfloat16: BF16, torch.float32: F32, torch.uint8: E4M3, torch.float8_e4m3fn: E4M3}
    d = GemmDesc()
    d.M = A.shape[0] if M is None else M
    d.N = Cout.shape[1] if groups <= 1 else B.shape[0] // groups
    d.K = A.shape[1]
    d.a_dtype, d.b_dtype, d.c_dtype = dt[A.dtype], dt[B.dtype], dt[Cout.dtype]
    d.A, d.lda = A.data_ptr(), A.stride(0)
    d.B, d.ldb = B.data_ptr(), B.stride(0)
    d.C, d.ldc = Cout.data_ptr(), Cout.stride(0)
    d.sa = sa.data_ptr() if sa is not None else None
    d.ld_sa = sa.stride(0) if sa is not None else 0
    d.sb = sb.data_ptr() if sb is not None else None
    d.group_offsets = group_offsets.data_ptr() if group_offsets is not None else None
    d.groups = groups
    d.mode = mode
    d.b_early = int(b_early)
    return d


def biv_gemm_workspace(desc: GemmDesc) -> int:
    n = C.c_size_t(0)
    _check(load().biv_gemm_workspace(C.byref(desc), C.byref(n)), "biv_gemm_workspace")
    return n.value


_gemm_scratch: Dict[int, torch.Tensor] = {}


def gemm_scratch(nbytes: int, device=None) -> torch.Tensor:
    """A scratch workspace of at least nbytes (GEMM chunk partials, SSD
    intermediates), cached per device (for callers on one stream)."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    t = _gemm_scratch.get(dev.index)
    if t is None or t.numel() < nbytes:
        t = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        _gemm_scratch[dev.index] = t
    return t


def biv_gemm(desc: GemmDesc, ws: Optional[torch.Tensor] = None, stream=None):
    """ws: a workspace of biv_gemm_workspace(desc) bytes; when None and the
    plan needs one, a cached per-device scratch buffer is used."""
    if ws is None:
        need = biv_gemm_workspace(desc)
        if need:
            ws = gemm_scratch(need)
    _check(load().biv_gemm(C.byref(desc), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                           _stream(stream)), "biv_gemm")


def biv_act_quant_fp8(x, codes, scales, stream=None):
    _check(load().biv_act_quant_fp8(_p(x), _rs(x), x.shape[0], x.shape[1], _p(codes), _p(scales),
                                    _stream(stream)), "biv_act_quant_fp8")


def biv_silu_mul_quant_fp8(gate_up, codes, scales, stream=None):
    _check(load().biv_silu_mul_quant_fp8(_p(gate_up), _rs(gate_up), gate_up.shape[0],
                                         codes.shape[1], _p(codes), _p(scales), _stream(stream)),
           "biv_silu_mul_quant_fp8")


def biv_topk(scores, valid_len, k, idx, stream=None):
    _check(load().biv_topk(_p(scores), scores.stride(0), _p(valid_len), scores.shape[0],
                           scores.shape[1], k, _p(idx), _stream(stream)), "biv_topk")


def biv_router_topk(logits, k, idx, w, stream=None):
    _check(load().biv_router_topk(_p(logits), logits.stride(0), logits.shape[0], logits.shape[1], k,
                                  _p(idx), _p(w), _stream(stream)), "biv_router_topk")


def biv_moe_dispatch(idx, E, offsets, perm, src_row, stream=None):
    _check(load().biv_moe_dispatch(_p(idx), idx.shape[0], idx.shape[1], E, _p(offsets), _p(perm),
                                   _p(src_row), _stream(stream)), "biv_moe_dispatch")


def biv_gather_rows(src, perm, k_div, n, dst, stream=None):
    rb = src.shape[1] * src.element_size()
    _check(load().biv_gather_rows(_p(src), src.stride(0) * src.element_size(), _p(perm), k_div, n, rb,
                                  _p(dst), dst.stride(0) * dst.element_size(), _stream(stream)),
           "biv_gather_rows")


def biv_moe_combine(y, src_row, w, shared, out, stream=None):
    T, k = w.shape
    _check(load().biv_moe_combine(_p(y), _p(src_row), _p(w), _p(shared), _p(out), T, k, out.shape[1],
                                  _stream(stream)), "biv_moe_combine")


def biv_logprob(logits, target, lp, T=None, stream=None):
    T = logits.shape[0] if T is None else T
    _check(load().biv_logprob(_p(logits), logits.stride(0), _p(target), T, logits.shape[1], _p(lp),
                              _stream(stream)), "biv_logprob")


def biv_lm_head_logprob_workspace(M: int, V: int) -> int:
    n = C.c_size_t(0)
    _check(load().biv_lm_head_logprob_workspace(M, V, C.byref(n)), "biv_lm_head_logprob_workspace")
    return n.value


def biv_lm_head_logprob(h, W, target, lp, workspace, M=None, mode=0, stream=None):
    """lp[:M] = log-softmax of (h[:M] . W^T) at target[:M], without FP32 logits."""
    M = h.shape[0] if M is None else M
    _check(load().biv_lm_head_logprob(_p(h), h.stride(0), _p(W), W.stride(0), M, W.shape[0], h.shape[1],
                                      _p(target), mode, _p(lp), _p(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream)),
           "biv_lm_head_logprob")


def biv_ssd_workspace(desc: SSDDesc) -> int:
    n = C.c_size_t(0)
    _check(load().biv_ssd_workspace(C.byref(desc), C.byref(n)), "biv_ssd_workspace")
    return n.value


def biv_ssd_scan(desc: SSDDesc, stream=None):
    """When desc.workspace is unset and the call has many new rows, a cached
    per-device scratch buffer serves as the workspace (callers on one stream)."""
    if not desc.workspace:
        need = biv_ssd_workspace(desc)
        if need:
            ws = gemm_scratch(need)
            desc.workspace, desc.workspace_bytes = ws.data_ptr(), ws.numel()
    _check(load().biv_ssd_scan(C.byref(desc), _stream(stream)), "biv_ssd_scan")


def biv_causal_conv1d(desc: ConvDesc, stream=None):
    _check(load().biv_causal_conv1d(C.byref(desc), _stream(stream)), "biv_causal_conv1d")


def biv_gated_rmsnorm(y, z, w, out, eps, rows=None, stream=None):
    """y, z, out: 2-D bf16 views (rows of d); w bf16 [d]."""
    _bf16_ok(y, z, w, out)
    n = y.shape[0] if rows is None else rows
    _check(load().biv_gated_rmsnorm(_p(y), _rs(y), _p(z), _rs(z), _p(w), _p(out), _rs(out), n,
                                    y.shape[-1], eps, _stream(stream)), "biv_gated_rmsnorm")


def biv_nvfp4_dequant(codes, scales, out, stream=None):
    """codes uint8 [N, K/2] (packed), scales uint8 [N, K/16] (e4m3) -> out bf16 [N, K]."""
    N, K = out.shape
    _check(load().biv_nvfp4_dequant(_p(codes), _p(scales), N, K, _p(out), _stream(stream)),
           "biv_nvfp4_dequant")


def biv_gemm_nvfp4_workspace(M, N, K, c_dtype=BF16, mode=MODE_INVARIANT) -> int:
    n = C.c_size_t(0)
    _check(load().biv_gemm_nvfp4_workspace(M, N, K, c_dtype, mode, C.byref(n)),
           "biv_gemm_nvfp4_workspace")
    return n.value


def biv_gemm_nvfp4(A, codes, scales, Cout, M=None, mode=MODE_INVARIANT, ws=None, stream=None):
    """Cout[M, N] = A[M, K] . dequant(codes, scales)^T; ws: a workspace of
    biv_gemm_nvfp4_workspace bytes (a cached per-device scratch when None)."""
    M = A.shape[0] if M is None else M
    N, K = codes.shape[0], A.shape[1]
    cdt = F32 if Cout.dtype == torch.float32 else BF16
    need = biv_gemm_nvfp4_workspace(M, N, K, cdt, mode)
    if ws is None and need:
        ws = gemm_scratch(need)
    _check(load().biv_gemm_nvfp4(_p(A), A.stride(0), _p(codes), _p(scales), M, N, K, _p(Cout),
                                 Cout.stride(0), cdt, mode, _p(ws), ws.numel() if ws is not None else 0,
                                 _stream(stream)), "biv_gemm_nvfp4")


# ------------------------------------------------------------- backward --
def biv_rmsnorm_backward(x, w, dy, dx, dw, eps, ws=None, stream=None):
    """x bf16 [R, d], w bf16 [d], dy float32 [R, d] -> dx float32 [R, d], dw float32 [d]."""
    R, d = x.shape
    if ws is None:
        ws = gemm_scratch(R * d * 4)
    _check(load().biv_rmsnorm_backward(_p(x), x.stride(0), _p(w), _p(dy), dy.stride(0), _p(dx),
                                       dx.stride(0), _p(dw), R, d, float(eps), _p(ws), ws.numel(),
                                       _stream(stream)), "biv_rmsnorm_backward")


def biv_silu_mul_backward(gate_up, dy, dgate_up, stream=None):
    R, I = dy.shape
    _check(load().biv_silu_mul_backward(_p(gate_up), gate_up.stride(0), _p(dy), dy.stride(0),
                                        _p(dgate_up), dgate_up.stride(0), R, I, _stream(stream)),
           "biv_silu_mul_backward")


def biv_logprob_backward(logits, target, dlp, dz, stream=None):
    T, V = logits.shape
    _check(load().biv_logprob_backward(_p(logits), logits.stride(0), _p(target), _p(dlp), T, V, _p(dz),
                                       dz.stride(0), _stream(stream)), "biv_logprob_backward")


def biv_attention_backward(q, k, v, dout, q_pos, k_pos, scale, dq, dk, dv, stream=None):
    """One sequence: q, dout bf16 [Tq, Hq, D]; k, v bf16 [Tk, Hkv, D]."""
    Tq, Hq, D = q.shape
    ws = gemm_scratch(2 * Tq * Hq * 4)
    d = AttnBwdDesc()
    d.q, d.k, d.v, d.dout = (t.data_ptr() for t in (q, k, v, dout))
    d.dq, d.dk, d.dv = dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
    d.Tq, d.Tk, d.Hq, d.Hkv, d.D = Tq, k.shape[0], Hq, k.shape[1], D
    d.q_pos, d.k_pos, d.scale, d.workspace = q_pos.data_ptr(), k_pos.data_ptr(), float(scale), ws.data_ptr()
    _check(load().biv_attention_backward(C.byref(d), _stream(stream)), "biv_attention_backward")


# ---------------------------------------------------------- policy loss --
def _rows_ok(what, t, dtype, n, dev):
    """A contiguous vector of at least n values on device dev."""
    if t.get_device() == dev and t.dtype is dtype and t.numel() >= n and t.is_contiguous():
        return
    if t.get_device() != dev:
        raise ValueError(f"{what} must be on the current CUDA device")
    raise ValueError(f"{what} must be a contiguous {dtype} tensor of at least {n} values")


def biv_policy_loss_workspace(T: int, nseq: int) -> int:
    n = C.c_size_t(0)
    _check(load().biv_policy_loss_workspace(T, nseq, C.byref(n)), "biv_policy_loss_workspace")
    return n.value


def policy_desc(seq_start, adv, stats, workspace, T: int, mask=None, old_lp=None, ref_lp=None,
                clip_lo=0.2, clip_hi=0.2, dual_clip=0.0, kl_coef=0.0, ent_coef=0.0,
                reduce=LOSS_TOKEN_MEAN, norm=1.0, adv_per_row=None) -> PolicyDesc:
    """The part that biv_policy_loss and biv_policy_loss_logits share (see
    include/biv.h).  seq_start int32 [nseq + 1]; adv float32 [nseq] (one per
    sequence) or [T]; mask uint8 or bool [T]; old_lp, ref_lp float32 [T];
    stats float32 [8]; workspace uint8 of biv_policy_loss_workspace bytes.
    adv_per_row says which adv is.  None goes by its length, and by sequence
    where nseq == T: a caller whose batches may have as many rows as sequences,
    some of them empty, has to say."""
    dev, f32, keep = _device(), torch.float32, (seq_start, adv, stats, workspace, mask, old_lp, ref_lp)
    nseq, nadv = seq_start.numel() - 1, adv.numel()
    if nseq < 0:
        raise ValueError("seq_start needs at least one entry")
    if adv_per_row is None:
        adv_per_row = nadv != nseq
    if nadv != (T if adv_per_row else nseq):
        raise ValueError(f"adv must hold {nseq} (sequences) or {T} (rows) values, as adv_per_row says")
    _rows_ok("seq_start", seq_start, torch.int32, 1, dev)
    _rows_ok("adv", adv, f32, 0, dev)
    _rows_ok("stats", stats, f32, 8, dev)
    _rows_ok("workspace", workspace, torch.uint8, 0, dev)
    if mask is not None:
        _rows_ok("mask", mask, torch.bool if mask.dtype is torch.bool else torch.uint8, T, dev)
        mask = mask.data_ptr()
    if old_lp is not None:
        _rows_ok("old_lp", old_lp, f32, T, dev)
        old_lp = old_lp.data_ptr()
    if ref_lp is not None:
        _rows_ok("ref_lp", ref_lp, f32, T, dev)
        ref_lp = ref_lp.data_ptr()
    d = PolicyDesc(T, nseq, seq_start.data_ptr(), mask, old_lp, ref_lp, adv.data_ptr(), int(adv_per_row),
                   clip_lo, clip_hi, dual_clip, kl_coef, ent_coef, reduce, norm, stats.data_ptr(),
                   workspace.data_ptr(), workspace.numel())
    d.tensors = keep     # they live as long as the descriptor
    return d


def biv_policy_loss(desc: PolicyDesc, lp, dlp=None, stream=None):
    """lp float32 [T] -> dlp float32 [T] (or None: statistics only) and desc's stats."""
    dev = _device()
    _rows_ok("lp", lp, torch.float32, desc.T, dev)
    if dlp is not None:
        _rows_ok("dlp", dlp, torch.float32, desc.T, dev)
        dlp = dlp.data_ptr()
    _check(load().biv_policy_loss(C.byref(desc), lp.data_ptr(), dlp, _stream(stream)), "biv_policy_loss")


_F32, _BF16, _U8 = torch.float32, torch.bfloat16, torch.uint8
_FLOATS = {_F32: F32, _BF16: BF16}


def _matrix(what, t, T, V, dev):
    """(row stride, type) of a float32 or bf16 matrix of at least T rows of V values."""
    kind, steps, size = _FLOATS.get(t.dtype), t.stride(), t.shape
    if t.get_device() != dev:
        raise ValueError(f"{what} must be on the current CUDA device")
    if kind is None or len(steps) != 2 or size[0] < T or size[1] != V or (V > 1 and steps[1] != 1):
        raise ValueError(f"{what} must be a float32 or bf16 [T, V] tensor with rows of stride 1")
    # (one row: its stride says nothing, and may be below V)
    return (steps[0] if T > 1 else max(steps[0], V)), kind


def biv_policy_loss_logits(desc: PolicyDesc, logits, target, lp, entropy, dz=None, inv_temp=1.0,
                           stream=None):
    """logits float32 or bf16 [T, V] (rows of stride 1) -> lp, entropy float32
    [T] and dz float32 or bf16 [T, V] (None: no gradient; may be logits)."""
    dev, T = _device(), desc.T
    V = logits.size(1) if logits.dim() == 2 else -1
    ld, zt = _matrix("logits", logits, T, V, dev)
    pz, ldz, dt = None, 0, F32
    if dz is not None:
        ldz, dt = _matrix("dz", dz, T, V, dev)
        pz = dz.data_ptr()
    _rows_ok("target", target, torch.int32, T, dev)
    _rows_ok("lp", lp, torch.float32, T, dev)
    _rows_ok("entropy", entropy, torch.float32, T, dev)
    _check(load().biv_policy_loss_logits(
        C.byref(desc), logits.data_ptr(), ld, zt, target.data_ptr(), V, inv_temp, lp.data_ptr(),
        entropy.data_ptr(), pz, ldz, dt, _stream(stream)), "biv_policy_loss_logits")


# -------------------------------------------- cross entropy of the LM head --
def _head(h, W, target, T, dev):
    """The sizes and row strides of an LM head's h bf16 [>= T, K] and W bf16 [V, K]."""
    T = h.size(0) if T is None else T
    for what, t in (("h", h), ("W", W)):
        if t.dtype is not torch.bfloat16 or t.dim() != 2 or t.get_device() != dev or \
                (t.size(1) > 1 and t.stride(1) != 1):
            raise ValueError(f"{what} must be a bf16 matrix with rows of stride 1 on the current CUDA device")
    if h.size(1) != W.size(1) or not 0 <= T <= h.size(0):
        raise ValueError("h [T, K] and W [V, K] do not fit")
    _rows_ok("target", target, torch.int32, T, dev)
    V, K = W.shape
    return T, V, K, (h.stride(0) if h.size(0) > 1 else K), (W.stride(0) if V > 1 else K)


def _vector(what, t, T, dev):
    """The address of a float32 vector of at least T values, or 0."""
    if t is None:
        return 0
    if t.dtype is not _F32 or t.get_device() != dev or t.numel() < T or not t.is_contiguous():
        _rows_ok(what, t, _F32, T, dev)
    return t.data_ptr()


def biv_lm_head_loss_workspace(T: int, V: int) -> int:
    n = C.c_size_t(0)
    _check(load().biv_lm_head_loss_workspace(T, V, C.byref(n)), "biv_lm_head_loss_workspace")
    return n.value


def biv_lm_head_loss(h, W, target, lp, lse, stats, workspace, weight=None, dlp=None, dlse=None, z_coef=0.0,
                     reduce=LOSS_TOKEN_MEAN, norm=1.0, ignore_index=-100, T=None, stream=None):
    """Cross entropy of the head's logits h . W^T with its coefficients dlp, dlse
    for biv_lm_head_backward (see include/biv.h).  stats float32 [4]; workspace
    uint8 of biv_lm_head_loss_workspace bytes; T: rows of h (all of them)."""
    dev = _device()
    T, V, K, ldh, ldw = _head(h, W, target, T, dev)
    _rows_ok("stats", stats, torch.float32, 4, dev)
    _rows_ok("workspace", workspace, torch.uint8, 0, dev)
    d = _pack_loss(T, V, K, h.data_ptr(), ldh, W.data_ptr(), ldw, target.data_ptr(),
                   _vector("weight", weight, T, dev), ignore_index, z_coef, reduce, norm,
                   _vector("lp", lp, T, dev), _vector("lse", lse, T, dev), _vector("dlp", dlp, T, dev),
                   _vector("dlse", dlse, T, dev), stats.data_ptr(), workspace.data_ptr(), workspace.numel())
    _check(load().biv_lm_head_loss(d, _stream(stream)), "biv_lm_head_loss")


def biv_lm_head_backward_workspace(T: int, V: int, K: int, dh_dtype=torch.bfloat16, dw_dtype=torch.bfloat16) -> int:
    n = C.c_size_t(0)
    _check(load().biv_lm_head_backward_workspace(T, V, K, _FLOATS.get(dh_dtype, -1), _FLOATS.get(dw_dtype, -1),
                                                 C.byref(n)), "biv_lm_head_backward_workspace")
    return n.value


def biv_lm_head_backward(h, W, target, lse, dlp, dh, dW, workspace, dlse=None, accumulate=False, T=None,
                         stream=None):
    """dh [T, K] and dW [V, K] (float32 or bf16; either may be None) from the
    coefficients dlp, dlse of a loss of lp and lse; accumulate adds to dW."""
    dev = _device()
    T, V, K, ldh, ldw = _head(h, W, target, T, dev)
    (lddh, ht), (lddw, wt) = (K, BF16), (K, BF16)
    if dh is not None:
        lddh, ht = _matrix("dh", dh, T, K, dev)
    if dW is not None:
        lddw, wt = _matrix("dW", dW, V, K, dev)
    _rows_ok("workspace", workspace, torch.uint8, 0, dev)
    d = _pack_grad(T, V, K, h.data_ptr(), ldh, W.data_ptr(), ldw, target.data_ptr(),
                   _vector("lse", lse, T, dev), _vector("dlp", dlp, T, dev), _vector("dlse", dlse, T, dev),
                   0 if dh is None else dh.data_ptr(), lddh, ht,
                   0 if dW is None else dW.data_ptr(), lddw, wt,
                   int(accumulate), workspace.data_ptr(), workspace.numel())
    _check(load().biv_lm_head_backward(d, _stream(stream)), "biv_lm_head_backward")


# -------------------------------------------------- activations in 8 bits --
def _bf16_rows(what, t, rows, width, dev):
    """(address, row stride) of a bf16 matrix of at least `rows` rows; zeros for None."""
    if t is None:
        return 0, 0
    steps, size = t.stride(), t.shape
    if t.dtype is not _BF16 or t.get_device() != dev or len(steps) != 2 or size[1] != width or size[0] < rows or \
            (steps[1] != 1 and width > 1):
        if t.dtype is not _BF16:
            raise ValueError(f"{what} must be bf16")
        _matrix(what, t, rows, width, dev)
    return t.data_ptr(), (steps[0] if rows > 1 else max(steps[0], width))


def _codes_of(what, codes, scales, rows, width, groups, dev):
    """The addresses of 8-bit rows without gaps and of their scales; zeros for None."""
    if (codes is None) != (scales is None):
        raise ValueError(f"{what} and its scales go together")
    if codes is None:
        return 0, 0
    if codes.dtype is not _U8 or codes.get_device() != dev or codes.numel() < rows * width or not codes.is_contiguous():
        _rows_ok(what, codes, _U8, rows * width, dev)
    return codes.data_ptr(), _vector(what + "'s scales", scales, rows * groups, dev)


def biv_add_rmsnorm_fp8(x, residual, w, eps, residual_out=None, y=None, codes=None, scales=None, keep=None,
                        keep_scales=None, inv=None, stream=None):
    """RMSNorm of x + residual with 8-bit outputs: y bf16 and/or codes, scales of
    the normed rows; keep, keep_scales, inv for biv_rmsnorm_backward_fp8 (see
    include/biv.h).  residual may be None; residual_out None writes it in place."""
    dev = _device()
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    rows, d = x.shape
    g = (d + 127) // 128
    _rows_ok("w", w, torch.bfloat16, d, dev)
    px, xs = _bf16_rows("x", x, rows, d, dev)
    pr, rs = _bf16_rows("residual", residual, rows, d, dev)
    po, ros = _bf16_rows("residual_out", residual_out, rows, d, dev)
    py, ys = _bf16_rows("y", y, rows, d, dev)
    pc, ps = _codes_of("codes", codes, scales, rows, d, g, dev)
    pk, pks = _codes_of("keep", keep, keep_scales, rows, d, g, dev)
    desc = _pack_norm(px, xs, pr, rs, po, ros, w.data_ptr(), py, ys, pc, ps, pk, pks,
                       _vector("inv", inv, rows, dev), rows, d, eps)
    _check(load().biv_add_rmsnorm_fp8(desc, _stream(stream)), "biv_add_rmsnorm_fp8")


def biv_rmsnorm_backward_fp8_workspace(rows: int, d: int) -> int:
    n = C.c_size_t(0)
    _check(load().biv_rmsnorm_backward_fp8_workspace(rows, d, C.byref(n)), "biv_rmsnorm_backward_fp8_workspace")
    return n.value


def biv_rmsnorm_backward_fp8(keep, keep_scales, inv, w, dy, dx, dw, workspace, dres=None, accumulate=False,
                             stream=None):
    """dx [rows, d] (float32 or bf16) and dw float32 [d] from kept 8-bit rows; dres
    (of dx's type) is added to dx, accumulate adds to dw."""
    dev = _device()
    if dy.dim() != 2:
        raise ValueError("dy must be a matrix")
    rows, d = dy.shape
    pk, ps = _codes_of("keep", keep, keep_scales, rows, d, (d + 127) // 128, dev)
    dys, yt = _matrix("dy", dy, rows, d, dev)
    dxs, xt = _matrix("dx", dx, rows, d, dev)
    pr, rs = 0, 0
    if dres is not None:
        rs, rt = _matrix("dres", dres, rows, d, dev)
        if rt != xt:
            raise ValueError("dres must have dx's type")
        pr = dres.data_ptr()
    _rows_ok("w", w, torch.bfloat16, d, dev)
    _rows_ok("dw", dw, torch.float32, d, dev)
    _rows_ok("workspace", workspace, torch.uint8, 0, dev)
    desc = _pack_norm_bwd(pk, ps, _vector("inv", inv, rows, dev), w.data_ptr(), dy.data_ptr(), dys, yt, pr, rs,
                          dx.data_ptr(), dxs, xt, dw.data_ptr(), int(accumulate), rows, d, workspace.data_ptr(),
                          workspace.numel())
    _check(load().biv_rmsnorm_backward_fp8(desc, _stream(stream)), "biv_rmsnorm_backward_fp8")


def biv_silu_mul_keep_fp8(gate_up, y, keep, keep_scales, stream=None):
    """biv_silu_mul (y bf16 [rows, I] or None) that keeps gate_up in 8 bits: keep
    uint8 [rows, 2I], keep_scales float32 [rows, 2 ceil(I / 128)]."""
    dev = _device()
    if gate_up.dim() != 2 or gate_up.size(1) % 2:
        raise ValueError("gate_up must be a matrix of 2I columns")
    rows, I = gate_up.size(0), gate_up.size(1) // 2  # noqa: E741
    pg, gs = _bf16_rows("gate_up", gate_up, rows, 2 * I, dev)
    py, ys = _bf16_rows("y", y, rows, I, dev)
    pk, ps = _codes_of("keep", keep, keep_scales, rows, 2 * I, 2 * ((I + 127) // 128), dev)
    _check(load().biv_silu_mul_keep_fp8(pg, gs, py, ys, pk, ps, rows, I, _stream(stream)), "biv_silu_mul_keep_fp8")


def biv_silu_mul_backward_fp8(keep, keep_scales, dy, dgate_up, y=None, stream=None):
    """dgate_up [rows, 2I] from kept 8-bit rows and dy [rows, I] (each float32 or
    bf16); y bf16 [rows, I] gets the activation of the kept values."""
    dev = _device()
    if dy.dim() != 2:
        raise ValueError("dy must be a matrix")
    rows, I = dy.shape  # noqa: E741
    pk, ps = _codes_of("keep", keep, keep_scales, rows, 2 * I, 2 * ((I + 127) // 128), dev)
    dys, yt = _matrix("dy", dy, rows, I, dev)
    dgs, gt = _matrix("dgate_up", dgate_up, rows, 2 * I, dev)
    py, ys = _bf16_rows("y", y, rows, I, dev)
    _check(load().biv_silu_mul_backward_fp8(pk, ps, dy.data_ptr(), dys, yt, dgate_up.data_ptr(), dgs, gt, py, ys,
                                            rows, I, _stream(stream)), "biv_silu_mul_backward_fp8")


# ------------------------------------------------------- optimizer step --
def biv_opt_plan(tensors):
    """Checks and completes a ctypes array of OptTensor; returns (chunks, kinds)."""
    n, k = C.c_int64(0), C.c_int(0)
    _check(load().biv_opt_plan(tensors, len(tensors), C.byref(n), C.byref(k)), "biv_opt_plan")
    return n.value, k.value


def biv_grad_norm_workspace(chunks: int) -> int:
    n = C.c_size_t(0)
    _check(load().biv_grad_norm_workspace(chunks, C.byref(n)), "biv_grad_norm_workspace")
    return n.value


def biv_grad_norm(table, n: int, chunks: int, max_norm, out, ws, stream=None):
    """table: device copy (uint8) of n planned OptTensors; out float32 [4], zeros before the first call."""
    _check(load().biv_grad_norm(_p(table), n, chunks, float(max_norm), _p(out), _p(ws), ws.numel(),
                                _stream(stream)), "biv_grad_norm")


def biv_adamw(desc: AdamWDesc, stream=None):
    _check(load().biv_adamw(C.byref(desc), _stream(stream)), "biv_adamw")
