"""ctypes binding of libsmol (include/smol.h): argument marshalling only.

Every computation runs in the library's CUDA kernels.  Importing this module
loads ``libsmol.so`` from this package directory and raises ImportError if it
has not been built (``python -c "import __graft_entry__ as g; g.build()"``);
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from ctypes import POINTER, c_float, c_int, c_size_t, c_void_p
from typing import Dict, List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsmol.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "smol.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libsmol.so is not built ({LIB_PATH}); run __graft_entry__.build() first")
_lib = ctypes.CDLL(LIB_PATH)

OK = 0
ERR_INVALID_ARG, ERR_UNSUPPORTED_SHAPE, ERR_MISALIGNED, ERR_TOO_LONG = -1, -2, -3, -4
ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE, ERR_TIMEOUT = -5, -6, -7, -8
ERR_RANGE, ERR_INPUT = -9, -10
OP_BLOCK, OP_MODEL, OP_DECODE = 1, 2, 3
ACT_BF16, ACT_F32 = 0, 1
KV_BF16, KV_E4M3 = 0, 1


class Config(ctypes.Structure):
    # no_rope_layers / sliding_window: host int32 arrays of n_layers entries or
    # NULL (assigning a ctypes array to the field keeps it alive with the struct)
    _fields_ = [("hidden", c_int), ("n_heads", c_int), ("n_kv_heads", c_int), ("head_dim", c_int),
                ("intermediate", c_int), ("n_layers", c_int), ("vocab", c_int), ("max_pos", c_int),
                ("rms_eps", c_float), ("rope_theta", c_float),
                ("no_rope_layers", POINTER(ctypes.c_int32)), ("sliding_window", POINTER(ctypes.c_int32))]


class BlockWeights(ctypes.Structure):
    _fields_ = [(k, c_void_p) for k in ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "wgate",
                                       "wup", "wdown")]


class ModelWeights(ctypes.Structure):
    _fields_ = [("layers", POINTER(BlockWeights)), ("embed", c_void_p), ("final_norm", c_void_p)]


class _PagedCacheStruct(ctypes.Structure):
    _fields_ = ([(k, c_void_p) for k in ("k_pages", "v_pages", "k_scale", "v_scale", "page_table")]
                + [(k, c_int) for k in ("kv_dtype", "n_layers", "n_pages", "n_kv_heads", "page_size", "head_dim",
                                        "max_pages")])


class _ChunkStruct(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int), ("pos", c_void_p), ("row_start", c_void_p), ("n_new", c_void_p),
                ("rows", ctypes.c_longlong)]


class _Rows(ctypes.Structure):
    _fields_ = [("data", c_void_p)] + [(k, ctypes.c_longlong) for k in ("layer", "seq", "row", "head")]


_CFG = POINTER(Config)
_PC, _CK, _RW = POINTER(_PagedCacheStruct), POINTER(_ChunkStruct), POINTER(_Rows)
_SIGS = {
    "smol_packed_bytes": (c_size_t, [_CFG, c_int, c_int]),
    "smol_prepare_weights": (c_int, [_CFG, POINTER(ModelWeights), c_int, c_void_p, c_size_t, c_void_p]),
    "smol_workspace_bytes": (c_size_t, [_CFG, c_int, c_int, c_int]),
    "smol_block_forward": (c_int, [_CFG, c_void_p, c_int, c_void_p, c_void_p, c_int, c_int, c_int, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "smol_model_forward": (c_int, [_CFG, c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p,
                                   c_void_p, c_size_t, c_void_p]),
    "smol_block_forward_masked": (c_int, [_CFG, c_void_p, c_int, c_void_p, c_void_p, c_int, c_int, c_int,
                                          c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "smol_model_forward_masked": (c_int, [_CFG, c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p,
                                          c_void_p, c_size_t, c_void_p]),
    "smol_decode_step": (c_int, [_CFG, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "smol_workspace_status": (c_int, [c_void_p, c_void_p]),
    "smol_last_launch_count": (c_int, []),
    "smol_status_string": (ctypes.c_char_p, [c_int]),
    "smol_decode_step_noalloc": (c_int, [_CFG, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p,
                                         c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "smol_decode_noalloc_status": (c_int, [c_void_p]),
    "smol_set_wait_limit_ns": (None, [ctypes.c_ulonglong]),
    "smol_decode_next": (c_int, [_CFG, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int,
                                 c_void_p, c_void_p, c_void_p, c_float, c_int, c_float, c_int, c_void_p,
                                 c_void_p, c_void_p, c_size_t, c_void_p]),
    "smol_append_kv": (c_int, [_CFG, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p,
                               c_void_p]),
    "smol_prefill_cache_workspace_bytes": (c_size_t, [_CFG, c_int, c_int, c_int]),
    "smol_prefill_with_cache": (c_int, [_CFG, c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                        c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "smol_sample": (c_int, [c_void_p, c_int, c_int, ctypes.c_longlong, c_float, c_int, c_float, c_int,
                            c_void_p, c_void_p, c_void_p]),
    "smol_paged_append": (c_int, [_PC, _CK, _RW, _RW, c_void_p]),
    "smol_paged_read": (c_int, [_PC, _CK, _RW, _RW, c_void_p]),
    "smol_paged_workspace_bytes": (c_size_t, [_PC, c_int, c_int, c_int]),
    "smol_paged_attention": (c_int, [_PC, c_int, _CK, c_int, _RW, _RW, c_float, c_int, c_void_p, c_size_t,
                                     c_void_p]),
    "smol_prefill_paged_workspace_bytes": (c_size_t, [_CFG, _PC, c_int, c_int]),
    "smol_prefill_paged": (c_int, [_CFG, c_void_p, c_void_p, c_int, c_int, _PC, c_void_p, c_void_p, c_void_p,
                                   c_size_t, c_void_p]),
    "smol_verify_workspace_bytes": (c_size_t, [c_int, c_int]),
    "smol_verify_drafts": (c_int, [c_void_p, ctypes.c_longlong, c_void_p, c_void_p, c_void_p, ctypes.c_longlong,
                                   c_int, c_int, c_int, c_float, c_int, c_float, c_int, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "smol_profile_begin": (c_int, [ctypes.c_uint, c_int]),
    "smol_profile_end": (c_int, [POINTER(c_int), POINTER(c_float), c_int]),
}

# kernel kinds of smol_profile_begin (SMOL_K_*)
KERNEL_KINDS = ("embed", "rowstats", "qkv_gemm_rope", "flash_attention", "o_gemm_residual",
                "gateup_gemm_swiglu", "down_gemm_residual", "lm_head_gemm", "decode_attention", "other",
                "sample")
(K_EMBED, K_ROWSTATS, K_QKV, K_ATTN, K_OPROJ, K_GATEUP, K_DOWN, K_HEAD, K_DEC_ATTN, K_OTHER,
 K_SAMPLE) = range(11)
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def declared_symbols() -> List[str]:
    """Function names declared in include/smol.h."""
    text = open(HEADER_PATH).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(smol_\w+)\s*\(", text, re.M)))


class SmolError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {code} ({status_string(code)})")


def status_string(code: int) -> str:
    return _lib.smol_status_string(code).decode()


def _check(code: int, where: str) -> None:
    if code != OK:
        raise SmolError(code, where)


def _i32_array(vals, n_layers: int, name: str):
    if vals is None:
        return None
    vals = [int(v) for v in vals]
    if len(vals) != n_layers:
        raise ValueError(f"{name} needs one entry per layer ({n_layers}), got {len(vals)}")
    return (ctypes.c_int32 * n_layers)(*vals)


def make_config(hidden, n_heads, n_kv_heads, head_dim, intermediate, n_layers, vocab, max_pos,
                rms_eps, rope_theta, no_rope_layers=None, sliding_window=None) -> Config:
    """no_rope_layers: per layer 1 = RoPE, 0 = NoPE block (None: RoPE everywhere);
    sliding_window: per layer 0 = full causal, w > 0 = window of w keys (None: none)."""
    cfg = Config(hidden, n_heads, n_kv_heads, head_dim, intermediate, n_layers, vocab, max_pos,
                 rms_eps, rope_theta)
    nr = _i32_array(no_rope_layers, n_layers, "no_rope_layers")
    sw = _i32_array(sliding_window, n_layers, "sliding_window")
    if nr is not None:
        cfg.no_rope_layers = nr
    if sw is not None:
        cfg.sliding_window = sw
    return cfg


def config_of(wl) -> Config:
    """Config from a synth.Workload (same field names)."""
    return make_config(wl.hidden, wl.n_heads, wl.n_kv_heads, wl.head_dim, wl.intermediate,
                       wl.n_layers, wl.vocab, wl.max_pos, wl.rms_eps, wl.rope_theta,
                       getattr(wl, "no_rope_layers", None), getattr(wl, "sliding_window", None))


def _p(t: Optional[torch.Tensor]):
    return None if t is None else c_void_p(t.data_ptr())


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _stream(stream=None):
    """The stream's handle: the given one's, else the current device's current stream's (without building a
    torch.cuda.Stream for it, which costs 3 us a call)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _dev(t: torch.Tensor, dtype, name: str) -> torch.Tensor:
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    return t


def packed_bytes(cfg: Config, n_layers: int, with_embed: bool) -> int:
    return _lib.smol_packed_bytes(ctypes.byref(cfg), n_layers, int(with_embed))


def workspace_bytes(cfg: Config, op: int, B: int, T: int) -> int:
    return _lib.smol_workspace_bytes(ctypes.byref(cfg), op, B, T)


def alloc_workspace(cfg: Config, op: int, B: int, T: int, device="cuda") -> torch.Tensor:
    n = workspace_bytes(cfg, op, B, T)
    if n == 0:
        raise SmolError(ERR_UNSUPPORTED_SHAPE, "smol_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


_LAYER_KEYS = ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "wgate", "wup", "wdown")


def prepare_weights(cfg: Config, layers: Sequence[Dict[str, torch.Tensor]], embed=None,
                    final_norm=None, stream=None) -> torch.Tensor:
    """Packs raw bf16 weights (device tensors) into a new device buffer."""
    n_layers = len(layers)
    arr = (BlockWeights * max(n_layers, 1))()
    for i, lw in enumerate(layers):
        arr[i] = BlockWeights(*[c_void_p(_dev(lw[k], torch.bfloat16, k).data_ptr()) for k in _LAYER_KEYS])
    mw = ModelWeights(arr, _p(embed), _p(final_norm))
    if embed is not None:
        _dev(embed, torch.bfloat16, "embed")
        _dev(final_norm, torch.bfloat16, "final_norm")
    n = packed_bytes(cfg, n_layers, embed is not None)
    if n == 0:
        raise SmolError(ERR_UNSUPPORTED_SHAPE, "smol_packed_bytes")
    device = embed.device if embed is not None else layers[0]["wq"].device
    packed = torch.empty(n, dtype=torch.uint8, device=device)
    _check(_lib.smol_prepare_weights(ctypes.byref(cfg), ctypes.byref(mw), n_layers, _p(packed), n,
                                     _stream(stream)), "smol_prepare_weights")
    return packed


def block_forward(cfg: Config, packed: torch.Tensor, layer: int, x: torch.Tensor, out: torch.Tensor,
                  ws: torch.Tensor, valid_start=None, k_out=None, v_out=None, stream=None) -> None:
    B, T, _ = x.shape
    if x.dtype not in (torch.bfloat16, torch.float32) or out.dtype != x.dtype:
        raise ValueError("x and out must both be bf16 or both fp32")
    _dev(x, x.dtype, "x")
    _dev(out, x.dtype, "out")
    act = ACT_F32 if x.dtype == torch.float32 else ACT_BF16
    if valid_start is not None:
        _dev(valid_start, torch.int32, "valid_start")
    _check(_lib.smol_block_forward(ctypes.byref(cfg), _p(packed), layer, _p(x), _p(out), act, B, T,
                                   _p(valid_start), _p(k_out), _p(v_out), _p(ws), ws.numel(),
                                   _stream(stream)), "smol_block_forward")


def block_forward_masked(cfg: Config, packed: torch.Tensor, layer: int, x: torch.Tensor, out: torch.Tensor,
                         ws: torch.Tensor, key_mask: torch.Tensor, k_out=None, v_out=None, stream=None) -> None:
    """block_forward with a key mask (uint8 [B, T], nonzero = visible) in place of left padding."""
    B, T, _ = x.shape
    if x.dtype not in (torch.bfloat16, torch.float32) or out.dtype != x.dtype:
        raise ValueError("x and out must both be bf16 or both fp32")
    _dev(x, x.dtype, "x")
    _dev(out, x.dtype, "out")
    _dev(key_mask, torch.uint8, "key_mask")
    if tuple(key_mask.shape) != (B, T):
        raise ValueError("key_mask must be [B, T]")
    act = ACT_F32 if x.dtype == torch.float32 else ACT_BF16
    _check(_lib.smol_block_forward_masked(ctypes.byref(cfg), _p(packed), layer, _p(x), _p(out), act, B, T,
                                          _p(key_mask), _p(k_out), _p(v_out), _p(ws), ws.numel(),
                                          _stream(stream)), "smol_block_forward_masked")


def model_forward_masked(cfg: Config, packed: torch.Tensor, ids: torch.Tensor, logits: torch.Tensor,
                         ws: torch.Tensor, key_mask: torch.Tensor, stream=None) -> None:
    """model_forward with a key mask (uint8 [B, T], nonzero = visible) in place of left padding."""
    B, T = ids.shape
    _dev(ids, torch.int32, "ids")
    _dev(logits, torch.bfloat16, "logits")
    _dev(key_mask, torch.uint8, "key_mask")
    if tuple(key_mask.shape) != (B, T):
        raise ValueError("key_mask must be [B, T]")
    _check(_lib.smol_model_forward_masked(ctypes.byref(cfg), _p(packed), _p(ids), B, T, _p(key_mask),
                                          _p(logits), _p(ws), ws.numel(), _stream(stream)),
           "smol_model_forward_masked")


def model_forward(cfg: Config, packed: torch.Tensor, ids: torch.Tensor, logits: torch.Tensor,
                  ws: torch.Tensor, valid_start=None, stream=None) -> None:
    B, T = ids.shape
    _dev(ids, torch.int32, "ids")
    _dev(logits, torch.bfloat16, "logits")
    _check(_lib.smol_model_forward(ctypes.byref(cfg), _p(packed), _p(ids), B, T, _p(valid_start),
                                   _p(logits), _p(ws), ws.numel(), _stream(stream)),
           "smol_model_forward")


def prefill_cache_workspace(cfg: Config, B: int, T: int, S_max: int, device="cuda") -> torch.Tensor:
    n = _lib.smol_prefill_cache_workspace_bytes(ctypes.byref(cfg), B, T, S_max)
    if n == 0:
        raise SmolError(ERR_UNSUPPORTED_SHAPE, "smol_prefill_cache_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def prefill_with_cache(cfg: Config, packed: torch.Tensor, ids: torch.Tensor, cache_len: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                       logits: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """T new tokens per sequence on top of a KV cache (chunked prefill)."""
    B, T = ids.shape
    S_max = k_cache.shape[3]
    _dev(ids, torch.int32, "ids")
    _dev(cache_len, torch.int32, "cache_len")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("k_new", k_new), ("v_new", v_new),
                    ("logits", logits)):
        _dev(t, torch.bfloat16, name)
    _check(_lib.smol_prefill_with_cache(ctypes.byref(cfg), _p(packed), _p(ids), B, T, _p(cache_len),
                                        _p(k_cache), _p(v_cache), S_max, _p(k_new), _p(v_new), _p(logits),
                                        _p(ws), ws.numel(), _stream(stream)), "smol_prefill_with_cache")


def decode_step(cfg: Config, packed: torch.Tensor, ids: torch.Tensor, cache_len: torch.Tensor,
                k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor,
                v_new: torch.Tensor, logits: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    B = ids.shape[0]
    S_max = k_cache.shape[3]
    _dev(ids, torch.int32, "ids")
    _dev(cache_len, torch.int32, "cache_len")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("k_new", k_new), ("v_new", v_new),
                    ("logits", logits)):
        _dev(t, torch.bfloat16, name)
    _check(_lib.smol_decode_step(ctypes.byref(cfg), _p(packed), _p(ids), _p(cache_len), B,
                                 _p(k_cache), _p(v_cache), S_max, _p(k_new), _p(v_new), _p(logits),
                                 _p(ws), ws.numel(), _stream(stream)), "smol_decode_step")


def decode_step_noalloc(cfg: Config, packed: torch.Tensor, ids: torch.Tensor, cache_len: torch.Tensor,
                        k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor,
                        v_new: torch.Tensor, logits: torch.Tensor, stream=None) -> None:
    """decode_step with the library's fixed device scratch instead of a workspace
    (for callers that cannot provide device memory; calls must not overlap)."""
    B = ids.shape[0]
    S_max = k_cache.shape[3]
    _dev(ids, torch.int32, "ids")
    _dev(cache_len, torch.int32, "cache_len")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("k_new", k_new), ("v_new", v_new),
                    ("logits", logits)):
        _dev(t, torch.bfloat16, name)
    _check(_lib.smol_decode_step_noalloc(ctypes.byref(cfg), _p(packed), _p(ids), _p(cache_len), B,
                                         _p(k_cache), _p(v_cache), S_max, _p(k_new), _p(v_new),
                                         _p(logits), _stream(stream)), "smol_decode_step_noalloc")


def decode_next(cfg: Config, packed: torch.Tensor, ids: torch.Tensor, cache_len: torch.Tensor,
                k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                next_ids: torch.Tensor, ws: torch.Tensor, logits: Optional[torch.Tensor] = None,
                uniform: Optional[torch.Tensor] = None, temperature: float = 1.0, top_k: int = 0,
                top_p: float = 1.0, do_sample: bool = False, stream=None) -> None:
    """The decode step and the next-token choice (greedy inside the head GEMM's
    epilogue; sampling through the choice kernel over `logits`)."""
    B = ids.shape[0]
    S_max = k_cache.shape[3]
    _dev(ids, torch.int32, "ids")
    _dev(cache_len, torch.int32, "cache_len")
    _dev(next_ids, torch.int32, "next_ids")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("k_new", k_new), ("v_new", v_new)):
        _dev(t, torch.bfloat16, name)
    if logits is not None:
        _dev(logits, torch.bfloat16, "logits")
    if uniform is not None:
        _dev(uniform, torch.float32, "uniform")
    _check(_lib.smol_decode_next(ctypes.byref(cfg), _p(packed), _p(ids), _p(cache_len), B, _p(k_cache),
                                 _p(v_cache), S_max, _p(k_new), _p(v_new), _p(logits), float(temperature),
                                 int(top_k), float(top_p), int(bool(do_sample)), _p(uniform), _p(next_ids),
                                 _p(ws), ws.numel(), _stream(stream)), "smol_decode_next")


def append_kv(cfg: Config, k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
              v_cache: torch.Tensor, cache_len: torch.Tensor, stream=None) -> None:
    """Appends a decode step's new keys/values at slot cache_len[b] and increments cache_len."""
    B = cache_len.shape[0]
    S_max = k_cache.shape[3]
    for name, t in (("k_new", k_new), ("v_new", v_new), ("k_cache", k_cache), ("v_cache", v_cache)):
        _dev(t, torch.bfloat16, name)
    _dev(cache_len, torch.int32, "cache_len")
    _check(_lib.smol_append_kv(ctypes.byref(cfg), B, _p(k_new), _p(v_new), _p(k_cache), _p(v_cache), S_max,
                               _p(cache_len), _stream(stream)), "smol_append_kv")


def sample(logits: torch.Tensor, next_ids: torch.Tensor, uniform: Optional[torch.Tensor] = None,
           temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, do_sample: bool = True,
           stream=None) -> None:
    """Next token of each row of logits [B, V] (bf16, rows may be strided) into
    next_ids [B] (int32); uniform [B] fp32 in [0, 1) unless greedy."""
    if logits.dim() != 2 or logits.dtype != torch.bfloat16 or not logits.is_cuda or logits.stride(1) != 1:
        raise ValueError("logits must be a CUDA bf16 [B, V] tensor with unit column stride")
    B, V = logits.shape
    _dev(next_ids, torch.int32, "next_ids")
    if uniform is not None:
        _dev(uniform, torch.float32, "uniform")
    _check(_lib.smol_sample(_p(logits), B, V, logits.stride(0), float(temperature), int(top_k),
                            float(top_p), int(bool(do_sample)), _p(uniform), _p(next_ids),
                            _stream(stream)), "smol_sample")


class PagedCache:
    """Descriptor of a key/value cache in pages (the tensors stay the caller's).

    k_pages, v_pages  [n_layers, n_pages, n_kv_heads, page_size, head_dim], bf16 or float8_e4m3fn
    page_table        int32 [B, max_pages]
    k_scale, v_scale  fp32 [n_layers, n_pages, n_kv_heads, page_size] with float8_e4m3fn pages
    """

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, k_scale=None,
                 v_scale=None):
        dtype = k_pages.dtype
        if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("pages must be bfloat16 or float8_e4m3fn")
        _dev(k_pages, dtype, "k_pages")
        _dev(v_pages, dtype, "v_pages")
        _dev(page_table, torch.int32, "page_table")
        if k_pages.dim() != 5 or v_pages.shape != k_pages.shape or page_table.dim() != 2:
            raise ValueError("pages must be [n_layers, n_pages, n_kv_heads, page_size, head_dim], page_table [B, max_pages]")
        self.e4m3 = dtype == torch.float8_e4m3fn
        if self.e4m3:
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if t is None or t.shape != k_pages.shape[:-1]:
                    raise ValueError(f"{name} must be [n_layers, n_pages, n_kv_heads, page_size] with float8_e4m3fn pages")
                _dev(t, torch.float32, name)
        elif k_scale is not None or v_scale is not None:
            raise ValueError("bfloat16 pages have no scales")
        self.tensors = (k_pages, v_pages, page_table, k_scale, v_scale)   # kept alive with the descriptor
        self.device = k_pages.device
        if any(t is not None and t.device != self.device for t in self.tensors):
            raise ValueError("pages, scales and page_table must be on one device")
        self.n_layers, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k_pages.shape
        self.n_seqs, self.max_pages = page_table.shape
        self.struct = _PagedCacheStruct(k_pages.data_ptr(), v_pages.data_ptr(),
                                        k_scale.data_ptr() if self.e4m3 else None,
                                        v_scale.data_ptr() if self.e4m3 else None, page_table.data_ptr(),
                                        KV_E4M3 if self.e4m3 else KV_BF16, self.n_layers, self.n_pages,
                                        self.n_kv_heads, self.page_size, self.head_dim, self.max_pages)
        self.ref = ctypes.byref(self.struct)


class Chunk:
    """Descriptor of a chunk of rows: row t of sequence b stands at position pos[b] + t.

    B, T       sequences, and the most rows that any has
    pos        int32 [B]
    row_start  int32 [B + 1]: the row tensors are packed, [rows, heads, head_dim], sequence b's rows at
               row_start[b] .. row_start[b + 1] - 1; None: they are [B, T, heads, head_dim]
    n_new      int32 [B] or None: rows of each sequence, without row_start (None: T)
    """

    def __init__(self, B: int, T: int, pos: torch.Tensor, row_start: Optional[torch.Tensor] = None,
                 n_new: Optional[torch.Tensor] = None):
        for name, t, n in (("pos", pos, B), ("row_start", row_start, B + 1), ("n_new", n_new, B)):
            if t is not None:
                _dev(t, torch.int32, name)
                if t.shape != (n,) or t.device != pos.device:
                    raise ValueError(f"{name} must be [{n}], on the device of pos")
        if row_start is not None and n_new is not None:
            raise ValueError("row_start and n_new exclude each other")
        self.tensors = (pos, row_start, n_new)
        self.B, self.T, self.packed, self.device = B, T, row_start is not None, pos.device
        self._fields = (B, T, pos.data_ptr(), None if row_start is None else row_start.data_ptr(),
                        None if n_new is None else n_new.data_ptr())
        self._ref = ctypes.byref(_ChunkStruct(*self._fields, 0))

    def ref(self, rows: int):
        """The C descriptor; of a packed chunk a new one, for tensors of `rows` rows."""
        return ctypes.byref(_ChunkStruct(*self._fields, rows)) if self.packed else self._ref


@functools.lru_cache(maxsize=1024)
def _row_strides(shape, strides, lead, n_layers, packed, B, T, heads, hd):
    """(layer, seq, row, head) strides of bf16 rows of that layout; a text where it does not fit."""
    if strides[-1] != 1:
        return "its last axis must be contiguous"
    if lead and shape[0] != n_layers:
        return f"it must have a first axis of {n_layers} layers"
    if shape[lead + (1 if packed else 2):] != (heads, hd) or (not packed and shape[lead:lead + 2] != (B, T)):
        return f"{tuple(shape)} does not fit the chunk ({heads} heads of {hd}, {'packed rows' if packed else (B, T)})"
    # the strides of axes of one entry say nothing (torch may give them any value)
    st = [s if n > 1 else hd for s, n in zip(strides[:-1], shape[:-1])]
    return st[0] if lead else hd, 0 if packed else st[lead], st[-2], st[-1]


def _rows(t: torch.Tensor, name: str, cache: PagedCache, chunk: Chunk, heads: int, lead: int) -> _Rows:
    """bf16 rows [(layers,) B, T, heads, head_dim], or [(layers,) rows, heads, head_dim] of a packed chunk."""
    if t.dtype != torch.bfloat16 or t.device != cache.device:
        raise ValueError(f"{name} must be bfloat16 on the cache's device")
    st = _row_strides(t.shape, t.stride(), lead, cache.n_layers, chunk.packed, chunk.B, chunk.T, heads, cache.head_dim)
    if isinstance(st, str):
        raise ValueError(f"{name}: {st}")
    return _Rows(t.data_ptr(), *st)


def _same_place(cache: PagedCache, chunk: Chunk) -> None:
    if chunk.device != cache.device or cache.device.index != torch.cuda.current_device():
        raise ValueError("the cache, the chunk and the current device must be one and the same")
    if chunk.B > cache.n_seqs:
        raise ValueError(f"{chunk.B} sequences, and {cache.n_seqs} rows of the page table")


def _here(*tensors) -> None:
    """All on the current device, where the call is going to run."""
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("every tensor must be on the current device")


def _paged_copy(fn, where, cache, chunk, k, v, names, stream):
    _same_place(cache, chunk)
    kr = _rows(k, names[0], cache, chunk, cache.n_kv_heads, 1)
    vr = _rows(v, names[1], cache, chunk, cache.n_kv_heads, 1)
    if k.shape != v.shape:
        raise ValueError(f"{names[0]} and {names[1]} must have the same rows")
    _check(fn(cache.ref, chunk.ref(k.shape[1]), ctypes.byref(kr), ctypes.byref(vr), _stream(stream)), where)


def paged_append(cache: PagedCache, chunk: Chunk, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
    """Writes a chunk's keys and values, [n_layers, B, T, n_kv_heads, head_dim] (any strides but the last) or
    [n_layers, rows, n_kv_heads, head_dim] packed, into the pages; e4m3 pages quantise them."""
    _paged_copy(_lib.smol_paged_append, "smol_paged_append", cache, chunk, k_new, v_new, ("k_new", "v_new"), stream)


def paged_read(cache: PagedCache, chunk: Chunk, k_out: torch.Tensor, v_out: torch.Tensor, stream=None) -> None:
    """The reverse of paged_append: the values at the chunk's positions into bf16 rows of the same layouts.
    `cache.transpose(2, 3)` of a dense [n_layers, B, n_kv_heads, S, head_dim] cache is such a layout."""
    _paged_copy(_lib.smol_paged_read, "smol_paged_read", cache, chunk, k_out, v_out, ("k_out", "v_out"), stream)


def alloc_paged_workspace(cache: PagedCache, n_heads: int, B: int, T: int) -> torch.Tensor:
    n = _lib.smol_paged_workspace_bytes(cache.ref, n_heads, B, T)
    if n == 0:
        raise SmolError(ERR_UNSUPPORTED_SHAPE, "smol_paged_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=cache.device)


def paged_attention(cache: PagedCache, layer: int, chunk: Chunk, q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                    scale: float = 0.0, window: int = 0, stream=None) -> None:
    """Causal grouped-query attention of a chunk of new tokens, already appended, over one layer of the cache.
    q, out: [B, T, n_heads, head_dim] or [rows, n_heads, head_dim] packed, bf16; scale 0: 1 / sqrt(head_dim)."""
    _same_place(cache, chunk)
    heads = q.shape[-2]
    qr = _rows(q, "q", cache, chunk, heads, 0)
    orr = _rows(out, "out", cache, chunk, heads, 0)
    if q.shape != out.shape:
        raise ValueError("q and out must have the same rows")
    if ws.device != cache.device:
        raise ValueError("ws must be on the cache's device")
    _check(_lib.smol_paged_attention(cache.ref, layer, chunk.ref(q.shape[0]), heads, ctypes.byref(qr), ctypes.byref(orr), scale,
                                     window, ws.data_ptr(), ws.numel(), _stream(stream)), "smol_paged_attention")


def prefill_paged_workspace(cfg: Config, cache: PagedCache, B: int, T: int) -> torch.Tensor:
    n = _lib.smol_prefill_paged_workspace_bytes(ctypes.byref(cfg), cache.ref, B, T)
    if n == 0:
        raise SmolError(ERR_UNSUPPORTED_SHAPE, "smol_prefill_paged_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=cache.device)


def prefill_paged(cfg: Config, packed: torch.Tensor, ids: torch.Tensor, cache: PagedCache, pos: torch.Tensor,
                  logits: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """T new tokens per sequence, ids [B, T], through the model over a paged cache, whose pages receive their keys
    and values; pos [B] (int32): tokens already there.  logits [B, T, V]."""
    B, T = ids.shape
    _dev(ids, torch.int32, "ids")
    _dev(pos, torch.int32, "pos")
    _dev(logits, torch.bfloat16, "logits")
    if pos.shape != (B,) or logits.shape != (B, T, cfg.vocab) or B > cache.n_seqs:
        raise ValueError("pos must be [B], logits [B, T, V], and the page table have B rows")
    _here(packed, ids, cache.tensors[0], pos, logits, ws)
    _check(_lib.smol_prefill_paged(ctypes.byref(cfg), packed.data_ptr(), ids.data_ptr(), B, T, cache.ref, pos.data_ptr(),
                                   logits.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)), "smol_prefill_paged")


def alloc_verify_workspace(B: int, T: int, device="cuda") -> torch.Tensor:
    n = _lib.smol_verify_workspace_bytes(B, T)
    if n == 0:
        raise SmolError(ERR_UNSUPPORTED_SHAPE, "smol_verify_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _table(t: torch.Tensor, name: str, dtype, shape, device: int) -> int:
    if not (t.get_device() == device and t.dtype == dtype and t.shape == shape and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on the current device")
    return t.data_ptr()


def _row_pitch(t: torch.Tensor, name: str, dtype, B: int, rows: int, V: int) -> int:
    """Elements from row to row of a [B, rows, V] tensor whose B * rows rows are evenly spaced."""
    if not (t.is_cuda and t.dtype == dtype and t.shape == (B, rows, V)):
        raise ValueError(f"{name} must be a CUDA {dtype} tensor of shape {(B, rows, V)}")
    s0, s1, s2 = t.stride()
    pitch = s1 if rows > 1 else s0 if B > 1 else V
    if (s2 != 1 and V > 1) or pitch < V or (B > 1 and s0 != rows * pitch):
        raise ValueError(f"{name}: rows must be contiguous and evenly spaced")
    return pitch


def verify_drafts(logits: torch.Tensor, drafts: torch.Tensor, n_accepted: torch.Tensor, next_ids: torch.Tensor,
                  ws: torch.Tensor, uniform: Optional[torch.Tensor] = None, draft_probs: Optional[torch.Tensor] = None,
                  n_draft: Optional[torch.Tensor] = None, p_draft: Optional[torch.Tensor] = None,
                  temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, do_sample: bool = True,
                  stream=None) -> None:
    """How many of each sequence's drafts [B, T] (int32) stay, and its next token, from the target's logits
    [B, T + 1, V] (bf16), the drafter's probabilities [B, T, V] (fp32; None: it chooses for certain) and
    uniform [B, T + 1] (fp32): column i decides draft i, the last one draws the next token.  No output may share
    memory with another tensor of the call."""
    B, T = drafts.shape
    V = logits.shape[-1]
    ld = _row_pitch(logits, "logits", torch.bfloat16, B, T + 1, V)
    ldq = 0 if draft_probs is None else _row_pitch(draft_probs, "draft_probs", torch.float32, B, T, V)
    _here(logits, draft_probs, ws)
    i32, f32, dev = torch.int32, torch.float32, logits.get_device()
    _check(_lib.smol_verify_drafts(
        logits.data_ptr(), ld, _table(drafts, "drafts", i32, (B, T), dev),
        None if n_draft is None else _table(n_draft, "n_draft", i32, (B,), dev),
        None if draft_probs is None else draft_probs.data_ptr(), ldq, B, T, V, temperature, top_k, top_p,
        int(bool(do_sample)), None if uniform is None else _table(uniform, "uniform", f32, (B, T + 1), dev),
        _table(n_accepted, "n_accepted", i32, (B,), dev), _table(next_ids, "next_ids", i32, (B,), dev),
        None if p_draft is None else _table(p_draft, "p_draft", f32, (B, T), dev), ws.data_ptr(), ws.numel(),
        _stream(stream)), "smol_verify_drafts")


def set_wait_limit_ns(ns: int) -> None:
    """Failure-path tests only: bounded-wait limit of the prefill and paged
    attention kernels for later launches (0 restores the default of 1 s)."""
    _lib.smol_set_wait_limit_ns(int(ns))


def decode_noalloc_status(stream=None) -> int:
    """Synchronising read (and reset) of the status word of decode_step_noalloc."""
    return _lib.smol_decode_noalloc_status(_stream(stream))


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronising read (and reset) of the kernels' status word."""
    return _lib.smol_workspace_status(_p(ws), _stream(stream))


def last_launch_count() -> int:
    return _lib.smol_last_launch_count()


def profile_begin(kind_mask: int, capacity: int) -> None:
    """Start per-launch event timing of the kernel kinds in kind_mask."""
    _check(_lib.smol_profile_begin(kind_mask, capacity), "smol_profile_begin")


def profile_end(cap: int = 65536):
    """Stop timing; returns [(kind, milliseconds), ...] in launch order."""
    kinds = (c_int * cap)()
    ms = (c_float * cap)()
    n = _lib.smol_profile_end(kinds, ms, cap)
    if n < 0:
        raise SmolError(n, "smol_profile_end")
    return [(kinds[i], ms[i]) for i in range(n)]


raw = _lib   # the C entry points themselves, for callers that marshal by hand
