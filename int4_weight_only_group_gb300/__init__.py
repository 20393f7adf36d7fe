"""GB300 int4 weight-only, group-wise decode step — Python binding of libkmr.

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of ``_lib/libkmr.so`` behind the C ABI declared in ``include/kmr.h``.
PyTorch is used only for device memory and streams.  There is no fallback:
if the library has not been built, every call raises ``KmrLibraryMissing``.

Names follow the C ABI (``kmr_pack_int4``, ``kmr_int4_gemv``,
``kmr_decode_attn``, ``kmr_decode_step`` ...).  Arrays may be numpy arrays
(host memory), torch tensors (host or device; their data pointer is passed)
or raw integer addresses.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

__all__ = [
    "KmrError", "KmrLibraryMissing", "lib", "library_path", "EXPORTED_SYMBOLS",
    "KMR_OK", "KMR_ERR_INVALID_ARG", "KMR_ERR_SHAPE", "KMR_ERR_SLOT_RANGE", "KMR_ERR_CACHE_FULL",
    "KMR_ERR_NO_PACK", "KMR_ERR_CUDA", "KMR_ERR_DEVICE_TIMEOUT", "KMR_ERR_BUFFER_SIZE", "KMR_ERR_BATCH",
    "KMR_PACK_GATE_UP", "KMR_EPI_NONE", "KMR_EPI_RESIDUAL", "KMR_EPI_SILU_MUL",
    "KMR_W_QKV", "KMR_W_O", "KMR_W_GATE_UP", "KMR_W_DOWN", "KMR_N_INPUT", "KMR_N_POST", "KMR_N_Q", "KMR_N_K",
    "ModelConfig", "kmr_status_string", "kmr_layout_version", "kmr_packed_size", "kmr_pack_int4",
    "kmr_unpack_int4", "kmr_int4_gemv", "kmr_decode_attn_workspace_size",
    "kmr_decode_attn", "kmr_decode_attn_noalloc", "kmr_decode_attn_cascade_workspace_size",
    "kmr_decode_attn_cascade", "Kv4Cache", "kmr_kv4_append", "kmr_kv4_from_bf16", "kmr_kv4_to_bf16",
    "kmr_decode_attn_kv4_workspace_size", "kmr_decode_attn_kv4", "kmr_kv4_evict", "KMR_F32", "KMR_BF16", "kmr_moe_route",
    "Moe", "kmr_moe_factors_size", "kmr_moe_prepare", "kmr_moe_experts_workspace_size", "kmr_moe_experts", "Lora", "kmr_lora_apply", "kmr_last_device_error", "kmr_smem_poison", "kmr_selftest_wait_timeout", "Model",
]

KMR_OK = 0
KMR_ERR_INVALID_ARG = -1
KMR_ERR_SHAPE = -2
KMR_ERR_SLOT_RANGE = -3
KMR_ERR_CACHE_FULL = -4
KMR_ERR_NO_PACK = -5
KMR_ERR_CUDA = -6
KMR_ERR_DEVICE_TIMEOUT = -7
KMR_ERR_BUFFER_SIZE = -8
KMR_ERR_BATCH = -9
KMR_PACK_GATE_UP = 1
KMR_EPI_NONE, KMR_EPI_RESIDUAL, KMR_EPI_SILU_MUL = 0, 1, 2
KMR_W_QKV, KMR_W_O, KMR_W_GATE_UP, KMR_W_DOWN = 0, 1, 2, 3
KMR_F32, KMR_BF16 = 0, 1
KMR_N_INPUT, KMR_N_POST, KMR_N_Q, KMR_N_K = 0, 1, 2, 3

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.path.join(_HERE, "_lib", "libkmr.so")


class KmrError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {kmr_status_string(code)} ({code})")


class KmrLibraryMissing(ImportError):
    pass


class ModelConfig(ctypes.Structure):
    """Mirror of kmr_model_config."""
    _fields_ = [
        ("hidden", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("intermediate", ctypes.c_int), ("vocab", ctypes.c_int),
        ("n_layers", ctypes.c_int), ("group", ctypes.c_int), ("eps", ctypes.c_float),
        ("rope_theta", ctypes.c_float), ("mrope_sections", ctypes.c_int * 3), ("qk_norm", ctypes.c_int),
        ("eos_id", ctypes.c_int), ("pad_id", ctypes.c_int), ("max_len", ctypes.c_int), ("slots", ctypes.c_int),
        ("max_batch", ctypes.c_int),
    ]


class Kv4CacheStruct(ctypes.Structure):
    """Mirror of kmr_kv4_cache."""
    _fields_ = [
        ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_sz", ctypes.c_void_p),
        ("v_sz", ctypes.c_void_p), ("slots", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("max_len", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("group", ctypes.c_int),
    ]


class MoeStruct(ctypes.Structure):
    """Mirror of kmr_moe."""
    _fields_ = [
        ("gate_up", ctypes.c_void_p), ("down", ctypes.c_void_p), ("experts", ctypes.c_int), ("hidden", ctypes.c_int),
        ("intermediate", ctypes.c_int), ("group", ctypes.c_int), ("factors", ctypes.c_void_p),
    ]


class LoraStruct(ctypes.Structure):
    """Mirror of kmr_lora."""
    _fields_ = [
        ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("adapters", ctypes.c_int), ("inputs", ctypes.c_int), ("outputs", ctypes.c_int), ("max_rank", ctypes.c_int),
    ]


_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
# name -> (restype, argtypes); every symbol include/kmr.h declares
_SIGNATURES = {
    "kmr_status_string": (ctypes.c_char_p, [_I]),
    "kmr_layout_version": (_I, []),
    "kmr_packed_size": (_SZ, [_I, _I, _I]),
    "kmr_pack_int4": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _SZ, _I, _P]),
    "kmr_unpack_int4": (_I, [_P, _SZ, _I, _I, _I, _I, _P, _P, _P, _I, _P]),
    "kmr_int4_gemv": (_I, [_P, _I, _I, _I, _I, _P, _I, _P, _I, _P]),
    "kmr_decode_attn_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "kmr_decode_attn": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _SZ, _P]),
    "kmr_decode_attn_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P]),
    "kmr_decode_attn_cascade_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "kmr_decode_attn_cascade": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _SZ,
                                     _P]),
    "kmr_kv4_append": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, ctypes.c_float, ctypes.c_float, _P, _P, _P,
                            _P]),
    "kmr_kv4_from_bf16": (_I, [_P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _I, _I, _P]),
    "kmr_kv4_to_bf16": (_I, [_P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _I, _I, _P]),
    "kmr_decode_attn_kv4_workspace_size": (_SZ, [_P, _I, _I, _I]),
    "kmr_decode_attn_kv4": (_I, [_P, _P, _P, _P, _I, _I, ctypes.c_float, _P, _P, _P, _SZ, _P]),
    "kmr_kv4_evict": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "kmr_moe_route": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "kmr_moe_factors_size": (_SZ, [_I, _I, _I]),
    "kmr_moe_prepare": (_I, [_P, _P]),
    "kmr_moe_experts_workspace_size": (_SZ, [_P, _I, _I, _I]),
    "kmr_moe_experts": (_I, [_P, _P, _I, _P, _P, _I, _I, _P, _I, _P, _SZ, _P]),
    "kmr_lora_apply": (_I, [_P, _P, _P, _P, _I, _P, _I, ctypes.c_longlong, ctypes.c_longlong, _P]),
    "kmr_last_device_error": (_I, []),
    "kmr_model_create": (_I, [ctypes.POINTER(ModelConfig), ctypes.POINTER(_P)]),
    "kmr_model_destroy": (_I, [_P]),
    "kmr_model_set_linear": (_I, [_P, _I, _I, _P, _P, _P]),
    "kmr_model_set_norm": (_I, [_P, _I, _I, _P]),
    "kmr_model_set_embedding": (_I, [_P, _P]),
    "kmr_model_set_kv": (_I, [_P, _I, _I, _I, _P, _P]),
    "kmr_model_kv_pointers": (_I, [_P, _I, ctypes.POINTER(_P), ctypes.POINTER(_P)]),
    "kmr_model_reserve_prefill": (_I, [_P, _I]),
    "kmr_prefill": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "kmr_model_copy_row_from": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _P]),
    "kmr_decode_step": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _P]),
    "kmr_decode_step_host": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _P]),
    "kmr_model_sync_status": (_I, [_P, _P]),
    "kmr_model_kernels_per_step": (_I, [_P, _I]),
    "kmr_model_device_bytes": (_SZ, [_P, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    "kmr_smem_poison": (_I, [ctypes.c_uint32, _P]),
    "kmr_selftest_wait_timeout": (_I, [ctypes.c_ulonglong, _P]),
    "kmr_model_set_smem_poison": (_I, [_P, _I, ctypes.c_uint32]),
    "kmr_model_set_prefill_tcgen05": (_I, [_P, _I]),
    "kmr_model_set_prefill_plan": (_I, [_P, _I, _I]),
    "kmr_prefill_plan": (_I, [_I, _I, _I, _I, _P, _P]),
    "kmr_model_set_persistent_step": (_I, [_P, _I]),
}
EXPORTED_SYMBOLS = tuple(_SIGNATURES)

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libkmr (raises KmrLibraryMissing if it was never built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise KmrLibraryMissing(f"{path} is missing: build it with int4_weight_only_group_gb300.build.build()")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


# ------------------------------------------------------------------ marshalling
def _ptr(a) -> Optional[int]:
    if a is None or type(a) is int:
        return a
    try:                                 # a contiguous torch.Tensor, at the least cost
        if a.is_contiguous():
            return a.data_ptr()
    except AttributeError:
        pass
    if isinstance(a, int):
        return a
    if hasattr(a, "data_ptr"):           # torch.Tensor
        if not a.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return a.data_ptr()
    if hasattr(a, "ctypes"):             # numpy.ndarray
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError("array must be C-contiguous")
        return a.ctypes.data
    raise TypeError(f"cannot pass {type(a).__name__} as a pointer")


# torch types of the 4-bit cache's device arguments (bf16 also as its bits), filled by the first tensor that is passed
_F32, _I32, _BF16 = set(), set(), set()


def _dev(a, kind: set, name: str) -> Optional[int]:
    """Device address of an argument: an address or None as it is, or a contiguous tensor of one of the types of `kind`.
    Sizes and devices are the caller's, as for the older calls: looking at types adds 0.2 us to the 15.5 us that an append and
    a conversion of one token take, looking at all three adds 4."""
    if a is None or type(a) is int:
        return a
    try:
        if a.dtype in kind and a.is_contiguous():
            return a.data_ptr()
    except AttributeError:
        pass
    return _dev_refused(a, kind, name)


def _learn_types() -> bool:
    """Fills the types' sets; whether they were empty."""
    import torch
    if _F32:
        return False
    _F32.add(torch.float32)
    _I32.add(torch.int32)
    _BF16.update((torch.bfloat16, torch.int16, torch.uint16))
    return True


def _dev_refused(a, kind, name):
    import torch
    if _learn_types():
        return _dev(a, kind, name)
    if isinstance(a, int):
        return int(a)
    if not isinstance(a, torch.Tensor):
        raise TypeError(f"cannot pass {type(a).__name__} as {name}")
    if a.dtype not in kind:
        raise ValueError(f"{name} is {a.dtype}: {' or '.join(sorted(map(str, kind)))} is needed")
    raise ValueError(f"{name} must be contiguous")


def _stream(s) -> Optional[int]:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream                  # torch.cuda.Stream


def _torch_stream(s, device):
    """The torch stream of a stream argument (None for tensors that are on no CUDA device)."""
    import torch
    if device.type != "cuda":
        return None
    if s is None or s == 0:
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(s, device) if isinstance(s, int) else s


def _check(code: int, where: str) -> None:
    if code != KMR_OK:
        raise KmrError(code, where)


# ------------------------------------------------------------------ C ABI wrappers
def kmr_status_string(code: int) -> str:
    try:
        return lib().kmr_status_string(code).decode()
    except KmrLibraryMissing:
        return f"status {code}"


def kmr_layout_version() -> int:
    return lib().kmr_layout_version()


def kmr_packed_size(N: int, K: int, group: int = 128) -> int:
    return lib().kmr_packed_size(N, K, group)


def kmr_pack_int4(q, s, z, N, K, group, flags, packed, packed_bytes, on_device, stream=None) -> None:
    _check(lib().kmr_pack_int4(_ptr(q), _ptr(s), _ptr(z), N, K, group, flags, _ptr(packed), packed_bytes,
                               int(on_device), _stream(stream)), "kmr_pack_int4")


def kmr_unpack_int4(packed, packed_bytes, N, K, group, flags, q, s, z, on_device, stream=None) -> None:
    _check(lib().kmr_unpack_int4(_ptr(packed), packed_bytes, N, K, group, flags, _ptr(q), _ptr(s), _ptr(z),
                                 int(on_device), _stream(stream)), "kmr_unpack_int4")


def kmr_int4_gemv(packed, N, K, group, flags, x, M, y, epilogue, stream=None) -> None:
    _check(lib().kmr_int4_gemv(_ptr(packed), N, K, group, flags, _ptr(x), M, _ptr(y), epilogue, _stream(stream)),
           "kmr_int4_gemv")


def kmr_decode_attn_workspace_size(B, nq, nkv, d) -> int:
    return lib().kmr_decode_attn_workspace_size(B, nq, nkv, d)


def kmr_decode_attn(q, k_cache, v_cache, slot_ids, cache_position, B, nq, nkv, d, max_len, slots, scale, out,
                    workspace, workspace_bytes, stream=None) -> None:
    _check(lib().kmr_decode_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(slot_ids), _ptr(cache_position), B,
                                 nq, nkv, d, max_len, slots, float(scale), _ptr(out), _ptr(workspace),
                                 workspace_bytes, _stream(stream)), "kmr_decode_attn")


def kmr_decode_attn_noalloc(q, k_cache, v_cache, slot_ids, cache_position, B, nq, nkv, d, max_len, slots, scale,
                            out, stream=None) -> None:
    """kmr_decode_attn for callers that cannot allocate device memory: no workspace argument,
    the library's fixed device scratch is used instead (see include/kmr.h for its limit)."""
    _check(lib().kmr_decode_attn_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(slot_ids),
                                         _ptr(cache_position), B, nq, nkv, d, max_len, slots, float(scale),
                                         _ptr(out), _stream(stream)), "kmr_decode_attn_noalloc")


def kmr_decode_attn_cascade_workspace_size(B, nq, nkv, d, prefix_len) -> int:
    return lib().kmr_decode_attn_cascade_workspace_size(B, nq, nkv, d, prefix_len)


def kmr_decode_attn_cascade(q, k_cache, v_cache, slot_ids, cache_position, prefix_slot, prefix_len, B, nq, nkv, d,
                            max_len, slots, scale, out, workspace, workspace_bytes, stream=None) -> None:
    """Shared-prefix decode attention: row b attends [0, prefix_len) of cache row prefix_slot,
    then [prefix_len, cache_position[b]] of its own row (see include/kmr.h)."""
    _check(lib().kmr_decode_attn_cascade(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(slot_ids),
                                         _ptr(cache_position), prefix_slot, prefix_len, B, nq, nkv, d, max_len,
                                         slots, float(scale), _ptr(out), _ptr(workspace), workspace_bytes,
                                         _stream(stream)), "kmr_decode_attn_cascade")


class Kv4Cache:
    """A 4-bit KV cache (kmr_kv4_cache) over four device tensors that it keeps alive: codes uint8
    [slots, n_kv, max_len, d / 2] of K and V, scale words int32 [slots, n_kv, max_len, d / group]
    (layout: include/kmr.h)."""

    def __init__(self, k_codes, v_codes, k_sz, v_sz):
        slots, n_kv, max_len, half = k_codes.shape
        groups = k_sz.shape[-1]
        if groups < 1 or (2 * half) % groups:
            raise ValueError("the scale words' last dimension must divide the head size")
        for t, size, last in ((k_codes, 1, half), (v_codes, 1, half), (k_sz, 4, groups), (v_sz, 4, groups)):
            if tuple(t.shape) != (slots, n_kv, max_len, last) or t.element_size() != size or not t.is_contiguous():
                raise ValueError("a 4-bit cache takes contiguous codes [slots, n_kv, max_len, d / 2] of one byte and "
                                 "scale words [slots, n_kv, max_len, d / group] of four")
            if t.device != k_codes.device:
                raise ValueError("the tensors of a 4-bit cache are on one device")
        self.tensors = (k_codes, v_codes, k_sz, v_sz)
        self.slots, self.n_kv_heads, self.max_len = slots, n_kv, max_len
        self.head_dim, self.group = 2 * half, 2 * half // groups
        self._struct = Kv4CacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_sz.data_ptr(), v_sz.data_ptr(), slots,
                                      n_kv, max_len, self.head_dim, self.group)
        self._as_parameter_ = ctypes.addressof(self._struct)

    @classmethod
    def zeros(cls, slots: int, n_kv_heads: int, max_len: int, head_dim: int, group: int = 32,
              device="cuda") -> "Kv4Cache":
        """A cache of its own, every value 0."""
        import torch
        codes = [torch.zeros((slots, n_kv_heads, max_len, head_dim // 2), dtype=torch.uint8, device=device)
                 for _ in range(2)]
        words = [torch.zeros((slots, n_kv_heads, max_len, head_dim // group), dtype=torch.int32, device=device)
                 for _ in range(2)]
        return cls(*codes, *words)

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.tensors)


_SECTIONS: dict = {}        # M-RoPE sections as C arrays (kept: the call reads them on the host)


def kmr_kv4_append(cache, qkv, positions, slot_ids, cache_position, n_tokens, B, T, nq, q_norm, k_norm, eps, rope_theta,
                   sections, q_out, mass=None, stream=None) -> None:
    """New tokens: q/k RMSNorm, M-RoPE, 4-bit K/V into the cache, rotated queries out (see include/kmr.h)."""
    sec = _SECTIONS.get(sections) if isinstance(sections, tuple) else None
    if sec is None:
        if len(sections) != 3:
            raise ValueError("three M-RoPE sections")
        sec = _SECTIONS[tuple(sections)] = (ctypes.c_int * 3)(*sections)
    _check(lib().kmr_kv4_append(cache, _dev(qkv, _F32, "qkv"), _dev(positions, _I32, "positions"), _dev(slot_ids, _I32, "slot_ids"),
                                _dev(cache_position, _I32, "cache_position"), _dev(n_tokens, _I32, "n_tokens"), B, T, nq,
                                _dev(q_norm, _BF16, "q_norm"), _dev(k_norm, _BF16, "k_norm"), eps, rope_theta, sec,
                                _dev(q_out, _F32, "q_out"), _dev(mass, _F32, "mass"), _stream(stream)), "kmr_kv4_append")


def kmr_kv4_from_bf16(cache, k_bf16, v_bf16, bf16_slots, bf16_max_len, bf16_slot_ids, bf16_start, slot_ids, start,
                      lengths, B, max_tokens, stream=None) -> None:
    """Spans of a bf16 cache into the 4-bit cache; the mass of a slot that was in use is the caller's to clear (see
    include/kmr.h)."""
    _check(lib().kmr_kv4_from_bf16(cache, _dev(k_bf16, _BF16, "k_bf16"), _dev(v_bf16, _BF16, "v_bf16"), bf16_slots, bf16_max_len,
                                   _dev(bf16_slot_ids, _I32, "bf16_slot_ids"), _dev(bf16_start, _I32, "bf16_start"),
                                   _dev(slot_ids, _I32, "slot_ids"), _dev(start, _I32, "start"), _dev(lengths, _I32, "lengths"),
                                   B, max_tokens, _stream(stream)), "kmr_kv4_from_bf16")


def kmr_kv4_to_bf16(cache, k_bf16, v_bf16, bf16_slots, bf16_max_len, bf16_slot_ids, bf16_start, slot_ids, start,
                    lengths, B, max_tokens, stream=None) -> None:
    """Spans of the 4-bit cache into a bf16 cache (see include/kmr.h)."""
    _check(lib().kmr_kv4_to_bf16(cache, _dev(k_bf16, _BF16, "k_bf16"), _dev(v_bf16, _BF16, "v_bf16"), bf16_slots, bf16_max_len,
                                 _dev(bf16_slot_ids, _I32, "bf16_slot_ids"), _dev(bf16_start, _I32, "bf16_start"),
                                 _dev(slot_ids, _I32, "slot_ids"), _dev(start, _I32, "start"), _dev(lengths, _I32, "lengths"),
                                 B, max_tokens, _stream(stream)), "kmr_kv4_to_bf16")


def kmr_decode_attn_kv4_workspace_size(cache, B, nq, with_mass=False) -> int:
    return lib().kmr_decode_attn_kv4_workspace_size(cache, B, nq, int(bool(with_mass)))


def kmr_decode_attn_kv4(cache, q, slot_ids, cache_position, B, nq, scale, mass, out, workspace, workspace_bytes,
                        stream=None) -> None:
    """Decode attention over the 4-bit cache; `mass` (or None) gains every position's weight (see include/kmr.h)."""
    _check(lib().kmr_decode_attn_kv4(cache, _dev(q, _F32, "q"), _dev(slot_ids, _I32, "slot_ids"),
                                     _dev(cache_position, _I32, "cache_position"), B, nq, scale, _dev(mass, _F32, "mass"),
                                     _dev(out, _F32, "out"), _ptr(workspace), workspace_bytes, _stream(stream)),
           "kmr_decode_attn_kv4")


def kmr_kv4_evict(src, dst, src_slot_ids, dst_slot_ids, lengths, B, keep, recent, mass, dst_mass, kept, new_lengths,
                  stream=None) -> None:
    """Cut rows to their newest and heaviest positions, compacted into other rows (see include/kmr.h)."""
    _check(lib().kmr_kv4_evict(src, dst, _dev(src_slot_ids, _I32, "src_slot_ids"), _dev(dst_slot_ids, _I32, "dst_slot_ids"),
                               _dev(lengths, _I32, "lengths"), B, keep, recent, _dev(mass, _F32, "mass"),
                               _dev(dst_mass, _F32, "dst_mass"), _dev(kept, _I32, "kept"), _dev(new_lengths, _I32, "new_lengths"),
                               _stream(stream)), "kmr_kv4_evict")


# ------------------------------------------------------------------ products whose weights each token chooses
def _act(dtype: int) -> set:
    """The tensor types of an activation argument."""
    return _BF16 if dtype == KMR_BF16 else _F32


class Moe:
    """An expert layer's weights (kmr_moe) over two device tensors that it keeps alive: the packed gate_up matrices
    (kmr_pack_int4 with KMR_PACK_GATE_UP) and the packed down matrices of `experts` MLPs, one behind the other.  They are
    packed before the object is made: kmr_moe_prepare runs here, on `stream`."""

    def __init__(self, gate_up, down, experts: int, hidden: int, intermediate: int, group: int = 128, stream=None):
        for t, name, size in ((gate_up, "gate_up", kmr_packed_size(2 * intermediate, hidden, group)),
                              (down, "down", kmr_packed_size(hidden, intermediate, group))):
            if size == 0:
                raise ValueError("hidden and intermediate are multiples of the group, which is 128")
            if t.element_size() != 1 or not t.is_contiguous() or t.numel() != experts * size:
                raise ValueError(f"{name} is not {experts} packed matrices of {size} bytes")
        if gate_up.device != down.device:
            raise ValueError("the tensors of an expert layer are on one device")
        import torch
        # memory of the stream that fills it: what is still queued on another one for a freed tensor's block does not reach it
        with torch.cuda.stream(_torch_stream(stream, gate_up.device)):
            factors = torch.empty(kmr_moe_factors_size(experts, hidden, intermediate), dtype=torch.uint8, device=gate_up.device)
        self.tensors = (gate_up, down, factors)
        self.experts, self.hidden, self.intermediate, self.group = experts, hidden, intermediate, group
        self._struct = MoeStruct(gate_up.data_ptr(), down.data_ptr(), experts, hidden, intermediate, group, factors.data_ptr())
        self._as_parameter_ = ctypes.addressof(self._struct)
        kmr_moe_prepare(self, stream)


class Lora:
    """Low-rank adapters of one projection (kmr_lora) over the device tensors a bf16 [adapters, max_rank, inputs],
    b bf16 [adapters, outputs, max_rank], ranks int32 [adapters] or None and scales fp32 [adapters] or None, kept alive."""

    def __init__(self, a, b, ranks=None, scales=None):
        adapters, rank, inputs = a.shape
        if b.dim() != 3 or b.shape[0] != adapters or b.shape[2] != rank:
            raise ValueError("adapters take a [adapters, max_rank, inputs] and b [adapters, outputs, max_rank]")
        for t in (ranks, scales):
            if t is not None and tuple(t.shape) != (adapters,):
                raise ValueError("ranks and scales have one value per adapter")
        if len({t.device for t in (a, b, ranks, scales) if t is not None}) > 1:
            raise ValueError("the tensors of the adapters are on one device")
        self.tensors = (a, b, ranks, scales)
        self.adapters, self.inputs, self.outputs, self.max_rank = adapters, inputs, b.shape[1], rank
        self._struct = LoraStruct(_dev(a, _BF16, "a"), _dev(b, _BF16, "b"), _dev(ranks, _I32, "ranks"),
                                  _dev(scales, _F32, "scales"), adapters, inputs, self.outputs, rank)
        self._as_parameter_ = ctypes.addressof(self._struct)


def _rows(a, kind: set, ld: int, name: str) -> Optional[int]:
    """Device address of rows that lie ld values apart: as _dev, or a matrix with that stride."""
    if a is None or type(a) is int:
        return a
    try:
        if a.dtype in kind and a.dim() == 2 and a.stride(1) == 1 and (a.shape[0] == 1 or a.stride(0) == ld):
            return a.data_ptr()
        if a.dtype in kind and a.dim() == 2:
            raise ValueError(f"{name} has rows {a.stride(0)} values apart (and values {a.stride(1)}), not {ld} (and 1)")
    except AttributeError:
        pass
    if not kind and _learn_types():              # (the first tensor of all)
        return _rows(a, kind, ld, name)
    return _dev(a, kind, name)


def kmr_moe_route(logits, dtype, T, experts, top_k, renormalise, ids, weights, stream=None) -> None:
    """Each token's top_k experts and their softmax weights (see include/kmr.h)."""
    _check(lib().kmr_moe_route(_dev(logits, _act(dtype), "logits"), dtype, T, experts, top_k, int(bool(renormalise)),
                               _dev(ids, _I32, "ids"), _dev(weights, _F32, "weights"), _stream(stream)), "kmr_moe_route")


def kmr_moe_factors_size(experts, hidden, intermediate) -> int:
    return lib().kmr_moe_factors_size(experts, hidden, intermediate)


def kmr_moe_prepare(moe, stream=None) -> None:
    """Fills the weights' factors (see include/kmr.h); Moe does so when it is made."""
    _check(lib().kmr_moe_prepare(moe, _stream(stream)), "kmr_moe_prepare")


def kmr_moe_experts_workspace_size(moe, dtype, T, top_k) -> int:
    return lib().kmr_moe_experts_workspace_size(moe, dtype, T, top_k)


def kmr_moe_experts(moe, x, dtype, ids, weights, T, top_k, y, epilogue, workspace, workspace_bytes, stream=None) -> None:
    """The weighted sum of each token's int4 experts (see include/kmr.h)."""
    kind = _act(dtype)
    _check(lib().kmr_moe_experts(moe, _dev(x, kind, "x"), dtype, _dev(ids, _I32, "ids"), _dev(weights, _F32, "weights"), T,
                                 top_k, _dev(y, kind, "y"), epilogue, _ptr(workspace), workspace_bytes, _stream(stream)),
           "kmr_moe_experts")


def kmr_lora_apply(lora, x, base, y, dtype, adapter_ids, T, ldx, ldy, stream=None) -> None:
    """base plus each row's low-rank adapter (see include/kmr.h).  x, base and y may be columns of wider matrices, whose
    rows lie ldx or ldy values apart."""
    kind = _act(dtype)
    _check(lib().kmr_lora_apply(lora, _rows(x, kind, ldx, "x"), _rows(base, kind, ldy, "base"), _rows(y, kind, ldy, "y"), dtype,
                                _dev(adapter_ids, _I32, "adapter_ids"), T, ldx, ldy, _stream(stream)), "kmr_lora_apply")


def kmr_prefill_plan(N: int, K: int, M: int, sms: int) -> Tuple[int, int]:
    """kmr_prefill_plan: (tokens per CTA, K split) of a tcgen05 prefill projection (host only)."""
    nt, ks = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().kmr_prefill_plan(int(N), int(K), int(M), int(sms), ctypes.byref(nt), ctypes.byref(ks)),
           "kmr_prefill_plan")
    return nt.value, ks.value


def kmr_last_device_error() -> int:
    return lib().kmr_last_device_error()


def kmr_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launch the bounded-wait self-test (a wait nothing completes gives up after limit_ns);
    kmr_last_device_error() then reads KMR_ERR_DEVICE_TIMEOUT."""
    _check(lib().kmr_selftest_wait_timeout(int(limit_ns), _stream(stream)), "kmr_selftest_wait_timeout")


def kmr_smem_poison(pattern: int, stream=None) -> None:
    """Fill every SM's shared memory with the 32-bit `pattern` (diagnostic; see include/kmr.h)."""
    _check(lib().kmr_smem_poison(pattern & 0xFFFFFFFF, _stream(stream)), "kmr_smem_poison")


# ------------------------------------------------------------------ model handle
class Model:
    """Owner of one kmr_model (packed weights, static KV cache, step scratch)."""

    def __init__(self, hidden, n_q_heads, n_kv_heads, head_dim, intermediate, vocab, n_layers, group=128,
                 eps=1e-6, rope_theta=1e6, mrope_sections: Sequence[int] = (16, 24, 24), qk_norm=True,
                 eos_id=-1, pad_id=0, max_len=1024, slots=1, max_batch=1):
        c = ModelConfig()
        c.hidden, c.n_q_heads, c.n_kv_heads, c.head_dim = hidden, n_q_heads, n_kv_heads, head_dim
        c.intermediate, c.vocab, c.n_layers, c.group = intermediate, vocab, n_layers, group
        c.eps, c.rope_theta = eps, rope_theta
        c.mrope_sections = (ctypes.c_int * 3)(*mrope_sections)
        c.qk_norm, c.eos_id, c.pad_id = int(bool(qk_norm)), eos_id, pad_id
        c.max_len, c.slots, c.max_batch = max_len, slots, max_batch
        self.config = c
        h = _P()
        _check(lib().kmr_model_create(ctypes.byref(c), ctypes.byref(h)), "kmr_model_create")
        self._h = h

    @classmethod
    def from_config(cls, cfg, max_batch: int = 1) -> "Model":
        """From any object with the ModelConfig field names (e.g. workloads.ModelConfig)."""
        return cls(cfg.hidden, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.intermediate, cfg.vocab,
                   cfg.n_layers, cfg.group, cfg.eps, cfg.rope_theta, tuple(cfg.mrope_sections), cfg.qk_norm,
                   cfg.eos_id, cfg.pad_id, cfg.max_len, cfg.slots, max_batch)

    @property
    def handle(self) -> int:
        return self._h.value

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().kmr_model_destroy(self._h)
            self._h = _P()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_linear(self, layer: int, which: int, q, s, z) -> None:
        _check(lib().kmr_model_set_linear(self._h, layer, which, _ptr(q), _ptr(s), _ptr(z)), "kmr_model_set_linear")

    def set_norm(self, layer: int, which: int, w) -> None:
        _check(lib().kmr_model_set_norm(self._h, layer, which, _ptr(w)), "kmr_model_set_norm")

    def set_embedding(self, e) -> None:
        _check(lib().kmr_model_set_embedding(self._h, _ptr(e)), "kmr_model_set_embedding")

    def set_kv(self, layer: int, slot: int, length: int, k, v) -> None:
        _check(lib().kmr_model_set_kv(self._h, layer, slot, length, _ptr(k), _ptr(v)), "kmr_model_set_kv")

    def kv_pointers(self, layer: int):
        k, v = _P(), _P()
        _check(lib().kmr_model_kv_pointers(self._h, layer, ctypes.byref(k), ctypes.byref(v)), "kmr_model_kv_pointers")
        return k.value, v.value

    def reserve_prefill(self, max_tokens: int) -> None:
        """kmr_model_reserve_prefill: scratch for prefill chunks of up to max_tokens positions."""
        _check(lib().kmr_model_reserve_prefill(self._h, max_tokens), "kmr_model_reserve_prefill")

    def prefill(self, token_ids, positions, T: int, slot: int, start_pos: int, state_token, state_positions,
                state_cache_position, state_finished, logits=None, stream=None) -> None:
        """kmr_prefill on device tensors: one prompt chunk into cache row `slot` at
        [start_pos, start_pos + T); the one-row state tensors receive the first decode step's state."""
        _check(lib().kmr_prefill(self._h, _ptr(token_ids), _ptr(positions), T, slot, start_pos, _ptr(state_token),
                                 _ptr(state_positions), _ptr(state_cache_position), _ptr(state_finished),
                                 _ptr(logits), _stream(stream)), "kmr_prefill")

    def copy_row_from(self, dst_slot: int, length: int, src_row: int, src_k=None, src_v=None, src_slots: int = 0,
                      src_max_len: int = 0, stream=None) -> None:
        """kmr_model_copy_row_from: positions [0, length) of row src_row of a source cache (device
        tensors or addresses of its layer 0, laid out like the model's cache; None: the model's own
        cache) into cache row dst_slot, every layer, K and V.  Queued on `stream`."""
        _check(lib().kmr_model_copy_row_from(self._h, dst_slot, _ptr(src_k), _ptr(src_v), src_slots, src_max_len,
                                             src_row, length, _stream(stream)), "kmr_model_copy_row_from")

    def decode_step(self, token_ids, positions, cache_position, slot_ids, finished, B: int, logits=None,
                    stream=None) -> None:
        """kmr_decode_step on device tensors (state advanced in place)."""
        _check(lib().kmr_decode_step(self._h, _ptr(token_ids), _ptr(positions), _ptr(cache_position),
                                     _ptr(slot_ids), _ptr(finished), B, _ptr(logits), _stream(stream)),
               "kmr_decode_step")

    def decode_step_host(self, token_ids, positions, cache_position, slot_ids, finished, B: int, logits=None,
                         stream=None) -> None:
        """kmr_decode_step_host on host arrays (copies in, steps, copies back, synchronises)."""
        _check(lib().kmr_decode_step_host(self._h, _ptr(token_ids), _ptr(positions), _ptr(cache_position),
                                          _ptr(slot_ids), _ptr(finished), B, _ptr(logits), _stream(stream)),
               "kmr_decode_step_host")

    def sync_status(self, stream=None) -> int:
        return lib().kmr_model_sync_status(self._h, _stream(stream))

    def kernels_per_step(self, B: int) -> int:
        return lib().kmr_model_kernels_per_step(self._h, B)

    def device_bytes(self) -> dict:
        """kmr_model_device_bytes: device memory the model holds, total and split."""
        w, kv, sc = _SZ(0), _SZ(0), _SZ(0)
        total = lib().kmr_model_device_bytes(self._h, ctypes.byref(w), ctypes.byref(kv), ctypes.byref(sc))
        return {"total": int(total), "weights": int(w.value), "kv_cache": int(kv.value), "scratch": int(sc.value)}

    def set_prefill_tcgen05(self, enable: bool) -> None:
        """kmr_model_set_prefill_tcgen05: run prefill projections on the tcgen05 kernel."""
        _check(lib().kmr_model_set_prefill_tcgen05(self._h, int(bool(enable))), "kmr_model_set_prefill_tcgen05")

    def set_prefill_plan(self, nt: int = 0, ksplit: int = 0) -> None:
        """kmr_model_set_prefill_plan: force the tcgen05 tile width / K split (0, 0: planned)."""
        _check(lib().kmr_model_set_prefill_plan(self._h, int(nt), int(ksplit)), "kmr_model_set_prefill_plan")

    def set_persistent_step(self, enable: bool) -> None:
        """kmr_model_set_persistent_step: run the step's layers as one persistent kernel."""
        _check(lib().kmr_model_set_persistent_step(self._h, int(bool(enable))), "kmr_model_set_persistent_step")

    def set_smem_poison(self, enable: bool, pattern: int = 0xFFFFFFFF) -> None:
        """Precede every kernel of the step with a shared-memory fill of `pattern` (diagnostic)."""
        _check(lib().kmr_model_set_smem_poison(self._h, int(bool(enable)), pattern & 0xFFFFFFFF),
               "kmr_model_set_smem_poison")
