"""The paged NVFP4 cache of keys and values as a decode loop holds it.

`KVCache` owns a layer's pool and the description the C ABI takes; `KVBatch` holds what a batch of
requests shares over its layers: block table, lengths, free pages, and the step's slots, which
`plan` makes on the GPU from the number of new tokens.  Codes and scales are those of QUADS §2.2
"FP4" (E2M1, one E4M3 scale per 16 elements of the head dimension), with one calibrated FP32
scale each for keys and values.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib as L


class _Desc(C.Structure):
    """nvq_kv_cache of include/nvfp4rac.h."""
    _fields_ = [("k_codes", C.c_void_p), ("k_sf", C.c_void_p), ("v_codes", C.c_void_p), ("v_sf", C.c_void_p),
                ("k_tscale", C.c_void_p), ("v_tscale", C.c_void_p), ("page_stride", C.c_int64), ("head_stride", C.c_int64),
                ("sf_page_stride", C.c_int64), ("sf_head_stride", C.c_int64), ("pages", C.c_int64), ("kv_heads", C.c_int32),
                ("page_size", C.c_int32), ("head_dim", C.c_int32)]


class KVCache:
    """Codes uint8 [pages, kv_heads, page_size, head_dim / 2], scales uint8 [pages, kv_heads, page_size,
    head_dim / 16] (keys and values alike; a page's rows contiguous, any strides between heads and
    pages), tensor scales float32 [1, 4] (nvq_tensor_scale)."""

    def __init__(self, k_codes, k_sf, v_codes, v_sf, k_tscale, v_tscale):
        pages, kv_heads, page_size, half = k_codes.shape
        rows = {"k_codes": (k_codes, half), "v_codes": (v_codes, half), "k_sf": (k_sf, half // 8), "v_sf": (v_sf, half // 8)}
        for name, (t, width) in rows.items():
            if t.shape != (pages, kv_heads, page_size, width) or t.stride()[2:] != (width, 1):
                raise ValueError(f"{name}: expected {(pages, kv_heads, page_size, width)} with contiguous page rows, got "
                                 f"{tuple(t.shape)}, strides {t.stride()}")
        if k_codes.stride() != v_codes.stride() or k_sf.stride() != v_sf.stride():
            raise ValueError("keys and values need the same strides")
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, kv_heads, page_size, 2 * half
        self.k_codes, self.k_sf, self.v_codes, self.v_sf = k_codes, k_sf, v_codes, v_sf
        self.k_tscale, self.v_tscale = k_tscale, v_tscale
        u8 = torch.uint8
        self._struct = _Desc(
            L._dev(k_codes, u8, "k_codes"), L._dev(k_sf, u8, "k_sf"), L._dev(v_codes, u8, "v_codes"), L._dev(v_sf, u8, "v_sf"),
            L._flat(k_tscale, torch.float32, "k_tscale", 4), L._flat(v_tscale, torch.float32, "v_tscale", 4),
            k_codes.stride(0), k_codes.stride(1), k_sf.stride(0), k_sf.stride(1), pages, kv_heads, page_size, 2 * half)
        self.desc = C.addressof(self._struct)

    @staticmethod
    def empty(pages: int, kv_heads: int, page_size: int, head_dim: int, k_amax: float, v_amax: float, device="cuda") -> "KVCache":
        """A pool whose scales cover magnitudes up to k_amax and v_amax (larger values saturate)."""
        def pool(width):
            return torch.zeros(pages, kv_heads, page_size, width, dtype=torch.uint8, device=device)
        return KVCache(pool(head_dim // 2), pool(head_dim // 16), pool(head_dim // 2), pool(head_dim // 16),
                       tensor_scale(k_amax, device), tensor_scale(v_amax, device))


def tensor_scale(amax: float, device="cuda") -> torch.Tensor:
    """The nvq_tensor_scale [1, 4] of a largest magnitude: S_enc = 2688 / amax, S_dec = 1 / S_enc in fp32."""
    a = torch.tensor(float(amax), dtype=torch.float32)
    if not torch.isfinite(a) or a < 0:
        raise ValueError(f"amax {amax} is not finite and non-negative")
    one = torch.ones((), dtype=torch.float32)
    s_enc = torch.clamp(torch.div(torch.full((), 2688.0), a), max=torch.finfo(torch.float32).max) if a > 0 else one
    t = torch.stack([a, s_enc, torch.div(one, s_enc), torch.zeros(())])
    if a > 0:
        t.view(torch.int32)[3] = int(torch.frexp(a).exponent) + 1  # ilogb(amax) + 2
    return t.view(1, 4).to(device)


class KVBatch:
    """Requests that decode together: `plan(new_tokens)` gives every new token its place."""

    def __init__(self, requests: int, page_size: int, max_len: int, pages: int, max_new: int, device="cuda"):
        """max_len: keys of the longest request; pages: of the pool; max_new: new tokens of a step."""
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = page_size
        self.block_table = torch.full((requests, -(-max_len // page_size)), -1, **i32)
        self.free_pages = torch.arange(pages - 1, -1, -1, **i32)  # page 0 is handed out first
        # the lengths and behind them the free count, and a place for the next step's: the plan's
        # outputs are not its inputs, and are copied over them, so that a captured plan advances
        self._held, self._next = (torch.zeros(requests + 1, **i32) for _ in range(2))
        self._held[requests] = pages
        self.kv_len, self.free_count = self._held[:requests], self._held[requests:]
        self._len_out, self._free_out = self._next[:requests], self._next[requests:]
        self.q_off = torch.zeros(requests + 1, **i32)
        self.slots = torch.full((max_new,), -1, dtype=torch.int64, device=device)
        self.positions = torch.full((max_new,), -1, **i32)
        self.workspace = torch.zeros(L.nvfp4_kv_attention_workspace_size(), dtype=torch.uint8, device=device)

    def plan(self, new_tokens: torch.Tensor, stream=None):
        """new_tokens int32 [requests]: fills q_off, slots and positions and advances kv_len and free_count, in the
        tensors that they are, so that each replay of a captured call is a step of its own."""
        if new_tokens.shape != self.kv_len.shape:
            raise ValueError(f"new_tokens: expected a count for each of {self.kv_len.numel()} requests, got {tuple(new_tokens.shape)}")
        L.nvfp4_kv_plan(new_tokens, self.kv_len, self.page_size, self.block_table, self.free_pages, self.free_count,
                        self._len_out, self._free_out, self.q_off, self.slots, positions=self.positions, stream=stream)
        with torch.cuda.stream(stream):
            self._held.copy_(self._next)
