"""ctypes binding of libhyper_attn.so (include/hyper_attn.h). Argument marshalling only.

The in-tree library is loaded on first use; if it is missing this raises instead of falling back to
anything else (build it with ``python -m approximate_long_context_b200.build`` or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# HA_LIBRARY=debug selects the HA_DEBUG build (bounds-checked index reads), any other value a library path
LIB_PATH = os.path.join(_HERE, "libhyper_attn.so")
if os.environ.get("HA_LIBRARY"):
    LIB_PATH = (os.path.join(_HERE, "libhyper_attn_debug.so") if os.environ["HA_LIBRARY"] == "debug"
                else os.environ["HA_LIBRARY"])

HA_OK, HA_ERR_INVALID_ARG, HA_ERR_UNSUPPORTED, HA_ERR_CUDA, HA_ERR_OOM, HA_ERR_TIMEOUT = 0, -1, -2, -3, -4, -5
DTYPES = {"bf16": 0, "fp32": 1}
KERNELS = {"auto": 0, "simt": 1, "tc": 2}
DBG = {"rank": 0, "near": 1, "perm": 2, "inv": 3, "lse": 4, "rn_s": 5, "rn_logw": 6}
SAMPLING = {"uniform": 0, "rownorm": 1}

# every symbol include/hyper_attn.h declares
EXPORTS = [
    "hyper_attn_create", "hyper_attn_set_options", "hyper_attn_default_options", "hyper_attn_forward",
    "hyper_attn_forward_host", "hyper_attn_draw", "hyper_attn_levels", "hyper_attn_debug_copy",
    "hyper_attn_status", "hyper_attn_last_launch_count", "hyper_attn_last_error", "hyper_attn_destroy",
    "hyper_attn_version", "hyper_attn_profile", "hyper_attn_profile_read",
    "hyper_attn_last_kernel", "hyper_attn_forward_noalloc", "hyper_attn_exact",
    "hyper_attn_diagnostics", "hyper_attn_backward", "hyper_attn_test_fail_alloc",
    "hyper_attn_prompt", "hyper_attn_prompt_workspace", "hyper_attn_tree", "hyper_attn_tree_workspace",
    "hyper_attn_cache_free", "hyper_attn_cache_fork", "hyper_attn_cache_workspace", "hyper_attn_cache_reserve",
    "hyper_attn_cache_append", "hyper_attn_cache_commit", "hyper_attn_capturing",
]
KERNEL_CLASSES = ["hash", "sort", "attn", "causal_base", "draws", "prompt", "tree", "cache"]


class HAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"hyper_attn error {code}: {msg}")
        self.code = code


class Options(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("batch", ctypes.c_int64),
        ("causal_base", ctypes.c_int64),
        ("stream", ctypes.c_void_p),
        ("kernel", ctypes.c_int),
        ("debug_captures", ctypes.c_int),
        ("bh_offset", ctypes.c_int64),
        ("test_stall_ms", ctypes.c_int),
        ("sampling", ctypes.c_int),
    ]


class PromptArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "o", "lse")] + [("tokens", ctypes.c_int64)] +
                [(n, ctypes.c_int64) for n in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head", "o_token",
                                               "o_head")] +
                [(n, ctypes.c_int) for n in ("heads", "kv_heads", "d")] +
                [("offsets", ctypes.c_void_p), ("seqs", ctypes.c_int64), ("max_len", ctypes.c_int64),
                 ("scale", ctypes.c_float), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)])


class CacheArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "table", "lens", "held", "refs")] +
                [(n, ctypes.c_int64) for n in ("layers", "pages", "slots", "max_pages")] +
                [(n, ctypes.c_int) for n in ("kv_heads", "page", "d")])


class TreeArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "o", "lse")] + [("tokens", ctypes.c_int64)] +
                [(n, ctypes.c_int64) for n in ("q_token", "q_head", "o_token", "o_head")] +
                [("heads", ctypes.c_int), ("layer", ctypes.c_int64)] +
                [(n, ctypes.c_void_p) for n in ("slots", "offsets", "mask")] +
                [("seqs", ctypes.c_int64), ("max_draft", ctypes.c_int), ("scale", ctypes.c_float),
                 ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)])


_lib = None


def lib():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: the CUDA library has not been built")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, u64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int
    L.hyper_attn_create.argtypes = [ctypes.POINTER(vp), ci]
    L.hyper_attn_set_options.argtypes = [vp, ctypes.POINTER(Options)]
    L.hyper_attn_default_options.argtypes = [ctypes.POINTER(Options)]
    L.hyper_attn_default_options.restype = None
    fwd = [vp, vp, vp, vp, vp, i64, ci, ci, ci, ci, ci, ci, u64]
    L.hyper_attn_forward.argtypes = fwd
    L.hyper_attn_forward_host.argtypes = fwd
    L.hyper_attn_exact.argtypes = [vp, vp, vp, vp, vp, i64, ci, ci, ci]
    L.hyper_attn_diagnostics.argtypes = [vp, vp, vp, i64, ci, ci, ci, ci, u64, i64, vp, vp]
    L.hyper_attn_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, ci, ci, ci, ci, ci, ci, u64]
    L.hyper_attn_test_fail_alloc.argtypes = [vp, ci]
    L.hyper_attn_draw.argtypes = [u64, ci, ci, i64, i64, ci, ci, i64, vp, vp]
    L.hyper_attn_levels.argtypes = [i64, ci, i64, ctypes.POINTER(ci), ctypes.POINTER(i64)]
    L.hyper_attn_debug_copy.argtypes = [vp, ci, ci, vp, ctypes.c_size_t]
    L.hyper_attn_status.argtypes = [vp]
    L.hyper_attn_last_launch_count.argtypes = [vp]
    L.hyper_attn_last_error.argtypes = [vp]
    L.hyper_attn_last_error.restype = ctypes.c_char_p
    L.hyper_attn_destroy.argtypes = [vp]
    L.hyper_attn_version.argtypes = []
    L.hyper_attn_profile.argtypes = [vp, ci]
    L.hyper_attn_last_kernel.argtypes = [vp]
    L.hyper_attn_forward_noalloc.argtypes = [vp, vp, vp, vp, i64, ci, ci, ci, ci, ci, u64, ci, vp]
    L.hyper_attn_profile_read.argtypes = [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ci), ci]
    st = ctypes.c_size_t
    L.hyper_attn_prompt.argtypes = [vp, ctypes.POINTER(PromptArgs)]
    L.hyper_attn_prompt_workspace.argtypes = [vp, i64, i64, i64, ci, ci]
    L.hyper_attn_prompt_workspace.restype = st
    L.hyper_attn_capturing.argtypes = [vp]
    cache = ctypes.POINTER(CacheArgs)
    L.hyper_attn_tree.argtypes = [vp, cache, ctypes.POINTER(TreeArgs)]
    L.hyper_attn_tree_workspace.argtypes = [vp, ci]
    L.hyper_attn_tree_workspace.restype = st
    L.hyper_attn_cache_free.argtypes = [vp, cache, vp, i64]
    L.hyper_attn_cache_fork.argtypes = [vp, cache, vp, vp, i64]
    L.hyper_attn_cache_workspace.argtypes = [i64, i64]
    L.hyper_attn_cache_workspace.restype = st
    L.hyper_attn_cache_reserve.argtypes = [vp, cache, vp, vp, i64, vp, vp, st]
    L.hyper_attn_cache_append.argtypes = [vp, cache, vp, vp, i64, i64, vp, vp, ctypes.c_char_p, ctypes.c_char_p, i64, i64]
    L.hyper_attn_cache_commit.argtypes = [vp, cache, vp, vp, vp, i64, i64]
    # the same entry points taking the argument struct as packed bytes
    L.prompt_packed = L["hyper_attn_prompt"]
    L.prompt_packed.argtypes = [vp, ctypes.c_char_p]
    L.tree_packed = L["hyper_attn_tree"]
    L.tree_packed.argtypes = [vp, cache, ctypes.c_char_p]
    _lib = L
    return L


def default_options() -> Options:
    o = Options()
    lib().hyper_attn_default_options(ctypes.byref(o))
    return o


def levels(n: int, causal: bool, base: int):
    L = ctypes.c_int()
    nodes = ctypes.c_int64()
    rc = lib().hyper_attn_levels(n, int(causal), base, ctypes.byref(L), ctypes.byref(nodes))
    if rc:
        raise HAError(rc, "invalid causal shape")
    return L.value, nodes.value


def draw(seed: int, d: int, r: int, bh: int, n: int, m: int, causal: bool = False, base: int = 4096):
    """The projection matrix (d, r) and samples (bh, nodes, m) the forward pass uses (host only)."""
    _, nodes = levels(n, causal, base) if causal else (0, 1)
    P = np.zeros((d, max(r, 1)), np.float32)
    S = np.zeros((bh, nodes, max(m, 1)), np.int32)
    rc = lib().hyper_attn_draw(seed, d, r, bh, n, m, int(causal), base, P.ctypes.data, S.ctypes.data)
    if rc:
        raise HAError(rc, "hyper_attn_draw failed")
    return P[:, :r].copy(), S[:, :, :m].copy()


def _ptr(x) -> int:
    if hasattr(x, "data_ptr"):
        if not x.is_contiguous():
            raise ValueError("tensors must be contiguous")
        return x.data_ptr()
    if isinstance(x, np.ndarray):
        if not x.flags["C_CONTIGUOUS"]:
            raise ValueError("arrays must be C-contiguous")
        return x.ctypes.data
    return int(x)


# The argument structs of the serving calls are packed with `struct` (native alignment): filling a ctypes Structure field by
# field takes several times as long, and these calls run once per layer and token.
_PROMPT = struct.Struct("@5Pq8q3iPqqfPN")
_TREE = struct.Struct("@3Pq4qiq3PqifPN")
_APPEND = struct.Struct("@3q")
_CACHE = struct.Struct("@6P4q3i4x")
_torch = None


def _import_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _ints(t, device: int, what: str, count=None, wide=False):
    """The address of a contiguous device tensor of int32 (wide: int64) values."""
    torch = _torch or _import_torch()
    if t.dtype is not (torch.int64 if wide else torch.int32) or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous int{64 if wide else 32} tensor on the handle's device is needed")
    if count is not None and t.numel() != count:
        raise ValueError(f"{what}: {count} values are needed, got {t.numel()}")
    return t.data_ptr()


class PagedCache:
    """A paged key/value cache in device tensors (ha_cache of the header): k, v [layers, pages, kv_heads, page, d],
    table [slots, max_pages], lens and held [slots], refs [pages] (int32). The tensors stay the caller's."""

    def __init__(self, k, v, table, lens, held, refs):
        shape, device = k.shape, k.get_device()
        if len(shape) != 5 or v.shape != shape or v.dtype is not k.dtype:
            raise ValueError("k and v: [layers, pages, kv_heads, page, d] of one type are needed")
        if not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("tensors must be contiguous")
        if device < 0 or v.get_device() != device:
            raise ValueError("the cache must be on one CUDA device")
        layers, pages, kv_heads, page, d = shape
        slots, max_pages = table.shape
        self.k, self.v, self.table, self.lens, self.held, self.refs = k, v, table, lens, held, refs
        self.device, self.dtype = device, k.dtype
        self.pages, self.kv_heads, self.page, self.d = pages, kv_heads, page, d
        self.args = CacheArgs.from_buffer_copy(_CACHE.pack(
            k.data_ptr(), v.data_ptr(), _ints(table, device, "table"), _ints(lens, device, "lens", slots),
            _ints(held, device, "held", slots), _ints(refs, device, "refs", pages), layers, pages, slots, max_pages, kv_heads,
            page, d))

    @classmethod
    def empty(cls, *, layers, pages, kv_heads, page, d, slots, max_pages, dtype="bf16", device=0):
        """A new cache with all pages free and all slots empty."""
        torch = _torch or _import_torch()
        dev = torch.device("cuda", device)
        shape = (layers, pages, kv_heads, page, d)
        kind = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
        return cls(torch.zeros(shape, dtype=kind, device=dev), torch.zeros(shape, dtype=kind, device=dev),
                   ints(slots, max_pages) - 1, ints(slots), ints(slots), ints(pages))


class HyperAttention:
    """One library handle bound to a CUDA device."""

    def __init__(self, device: int = 0):
        self._h = ctypes.c_void_p()
        rc = lib().hyper_attn_create(ctypes.byref(self._h), device)
        if rc:
            raise HAError(rc, f"hyper_attn_create(device={device}) failed")
        self.options = default_options()
        self.device = device
        self._device_object = None
        self._ws, self._ws_ptr, self._ws_bytes = None, 0, 0
        self._captured, self._pooled, self._pool_freed = [], set(), -1
        self._needs = {}

    def _check(self, rc: int):
        if rc:
            raise HAError(rc, lib().hyper_attn_last_error(self._h).decode())

    def set_options(self, *, dtype="bf16", out_dtype=None, batch=1, causal_base=4096, stream=None,
                    kernel="auto", debug_captures=False, bh_offset=0, test_stall_ms=0, sampling="uniform"):
        o = Options()
        o.dtype = DTYPES[dtype]
        o.out_dtype = -1 if out_dtype is None else DTYPES[out_dtype]
        o.batch = batch
        o.causal_base = causal_base
        o.stream = stream
        o.kernel = KERNELS[kernel]
        o.debug_captures = int(bool(debug_captures))
        o.bh_offset = bh_offset
        o.test_stall_ms = test_stall_ms
        o.sampling = SAMPLING[sampling]
        self._check(lib().hyper_attn_set_options(self._h, ctypes.byref(o)))
        if o.stream != self.options.stream:   # the buffer's reuse was ordered by the old stream
            self._ws, self._ws_ptr, self._ws_bytes = None, 0, 0
        self.options = o
        self._needs.clear()

    def forward(self, Q, K, V, O, *, n, d, heads, block, m, r, causal, seed):
        """Device tensors (torch CUDA tensors or raw device addresses)."""
        self._check(lib().hyper_attn_forward(self._h, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), n, d, heads, block, m, r,
                                             int(causal), seed))

    def exact(self, Q, K, V, O, *, n, d, heads, causal):
        """Exact softmax attention (device tensors) on the tensor-core kernel; enqueued on the handle's stream."""
        self._check(lib().hyper_attn_exact(self._h, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), n, d, heads, int(causal)))

    def backward(self, Q, K, V, dO, dQ, dK, dV, *, n, d, heads, block, m, r, causal, seed):
        """Gradients of sum(dO * O) into fp32 device tensors dQ, dK, dV (the forward is recomputed); enqueued on
        the handle's stream."""
        self._check(lib().hyper_attn_backward(self._h, _ptr(Q), _ptr(K), _ptr(V), _ptr(dO), _ptr(dQ), _ptr(dK),
                                              _ptr(dV), n, d, heads, block, m, r, int(causal), seed))

    def diagnostics(self, Q, K, *, n, d, heads, block, r, seed, first_col=0):
        """(alpha, kappa) arrays of length batch*heads for device tensors Q, K (synchronous)."""
        bh = self.options.batch * heads
        alpha = np.zeros(bh, np.float64)
        kappa = np.zeros(bh, np.float64)
        self._check(lib().hyper_attn_diagnostics(self._h, _ptr(Q), _ptr(K), n, d, heads, block, r, seed, first_col,
                                                 alpha.ctypes.data, kappa.ctypes.data))
        return alpha, kappa

    def forward_host(self, Q, K, V, O, *, n, d, heads, block, m, r, causal, seed):
        """Host buffers (numpy arrays or CPU torch tensors, preferably page-locked); blocks until O is ready."""
        self._check(lib().hyper_attn_forward_host(self._h, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), n, d, heads, block, m,
                                                  r, int(causal), seed))

    # ---- serving: exact attention over packed prompts and over a paged cache, and the cache's steps

    def _rows(self, t, what: str, dtype: int):
        """Address and strides of a [tokens, heads, d] device tensor of the given type with a contiguous last dimension."""
        torch = _torch or _import_torch()
        stride = t.stride()
        if len(stride) != 3 or (stride[2] != 1 and t.shape[2] != 1):
            raise ValueError(f"{what}: [tokens, heads, d] with contiguous rows is needed")
        if t.dtype is not (torch.float32 if dtype else torch.bfloat16):
            raise ValueError(f"{what}: the handle's options say {'fp32' if dtype else 'bf16'}, got {t.dtype}")
        if t.get_device() != self.device:
            raise ValueError(f"{what}: on the handle's device")
        return t.data_ptr(), stride[0], stride[1]

    def _need(self, ask, sizes) -> int:
        """The workspace of a call with these sizes under the options as they are; the library is asked once."""
        nbytes = self._needs.get(sizes)
        if nbytes is None:
            if len(self._needs) >= 256:
                self._needs.clear()
            nbytes = self._needs[sizes] = ask(self._h, *sizes)
        return nbytes

    def _workspace(self, nbytes: int) -> int:
        """The address of a device buffer of at least nbytes. Eager calls share one, in the order of the handle's stream; a
        call under capture gets its own, from the graph's memory."""
        if not nbytes:
            return 0
        capturing = _lib.hyper_attn_capturing(self._h)
        if nbytes <= self._ws_bytes and not capturing:
            return self._ws_ptr
        torch = _torch or _import_torch()
        stream = self.options.stream or 0
        if stream == torch.cuda.current_stream(self.device).cuda_stream:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self._torch_device())
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=self._torch_device()) if stream
                                   else torch.cuda.default_stream(self.device)):
                ws = torch.empty(nbytes, dtype=torch.uint8, device=self._torch_device())
        if not capturing:
            self._ws, self._ws_ptr, self._ws_bytes = ws, ws.data_ptr(), nbytes
        elif not self._in_graph_pool(ws.data_ptr()):
            self._captured.append(ws)   # a capture that torch does not know of: its memory is not the graph's
        return ws.data_ptr()

    def _in_graph_pool(self, ptr: int) -> bool:
        """Whether the memory at ptr is of one of torch's private pools, which a capture by torch allocates from and which lives
        as long as its graph. An answer holds until torch gives memory back to the device."""
        freed = _torch.cuda.memory_stats(self.device).get("segment.all.freed")
        if freed is None:
            return False                # another allocator than torch's own: nothing is known
        if freed != self._pool_freed:
            self._pool_freed = freed
            self._pooled.clear()
        if ptr not in self._pooled:
            for segment in _torch.cuda.memory_snapshot(include_traces=False):
                if 0 <= ptr - segment["address"] < segment["total_size"] and tuple(segment["segment_pool_id"]) != (0, 0):
                    self._pooled.add(ptr)
        return ptr in self._pooled

    def _torch_device(self):
        if self._device_object is None:
            self._device_object = (_torch or _import_torch()).device("cuda", self.device)
        return self._device_object

    def _out_dtype(self) -> int:
        out = self.options.out_dtype
        return self.options.dtype if out < 0 else out

    def _lse(self, lse, heads: int, tokens: int):
        if lse is None:
            return None
        if (lse.shape != (heads, tokens) or lse.dtype is not _torch.float32 or lse.get_device() != self.device or
                not lse.is_contiguous()):
            raise ValueError("lse: contiguous fp32 [heads, tokens] on the handle's device is needed")
        return lse.data_ptr()

    def prompt(self, Q, K, V, O, offsets, *, max_len=None, scale=1.0, lse=None):
        """Exact causal attention over packed prompts: Q, O [tokens, heads, d], K, V [tokens, kv_heads, d] device tensors
        (any token and head strides), offsets [seqs + 1] int32; lse [heads, tokens] fp32 is optional. No sequence is
        longer than max_len (default: tokens). Rows behind the last sequence are left as they are."""
        dt = self.options.dtype
        q, k, v = self._rows(Q, "Q", dt), self._rows(K, "K", dt), self._rows(V, "V", dt)
        o = self._rows(O, "O", self._out_dtype())
        tokens, heads, d = shape = Q.shape
        kshape = K.shape
        kv_heads = kshape[1]
        if O.shape != shape or V.shape != kshape or kshape[0] != tokens or kshape[2] != d:
            raise ValueError("Q, O [tokens, heads, d] and K, V [tokens, kv_heads, d] are needed")
        at = _ints(offsets, self.device, "offsets")
        seqs = offsets.numel() - 1
        L = _lib
        if max_len is None:
            max_len = max(tokens, 1)
        nbytes = self._need(L.hyper_attn_prompt_workspace, (tokens, seqs, max_len, heads, kv_heads))
        ws = self._workspace(nbytes)
        rc = L.prompt_packed(self._h, _PROMPT.pack(
            q[0], k[0], v[0], o[0], self._lse(lse, heads, tokens) or 0, tokens, q[1], q[2], k[1], k[2], v[1], v[2], o[1], o[2],
            heads, kv_heads, d, at, seqs, max_len, scale,
            ws, nbytes))
        if rc:
            self._check(rc)

    def _cache(self, cache):
        if cache.device != self.device:
            raise ValueError("the cache must be on the handle's device")
        if cache.dtype is not (_torch.float32 if self.options.dtype else _torch.bfloat16):
            raise ValueError(f"the cache holds {cache.dtype}, the handle's options say another type")
        return cache.args

    def tree(self, Q, cache, O, slots, offsets, *, mask=None, max_draft=64, layer=0, scale=1.0, lse=None):
        """Exact attention of drafted tokens (or single ones) over a PagedCache: sequence i (slot slots[i]; None: slot i) has
        the rows offsets[i] .. offsets[i+1]-1 of Q and O [tokens, heads, d], whose keys and values were appended behind
        the slot's committed rows. mask [tokens] int64: bit j of a row lets it see drafted row j (None: rows 0..i). max_draft:
        no sequence has more rows; the kernel is chosen by it, so a bound near the truth (1 for decoding) is the faster one."""
        c = self._cache(cache)
        q, o = self._rows(Q, "Q", self.options.dtype), self._rows(O, "O", self._out_dtype())
        tokens, heads, d = shape = Q.shape
        if O.shape != shape or d != cache.d:
            raise ValueError("Q, O [tokens, heads, d] with the cache's d are needed")
        at = _ints(offsets, self.device, "offsets")
        seqs = offsets.numel() - 1
        L = _lib
        nbytes = self._need(L.hyper_attn_tree_workspace, (d,))
        ws = self._workspace(nbytes)
        rc = L.tree_packed(self._h, c, _TREE.pack(
            q[0], o[0], self._lse(lse, heads, tokens) or 0, tokens, q[1], q[2], o[1], o[2], heads, layer,
            0 if slots is None else _ints(slots, self.device, "slots", seqs), at,
            0 if mask is None else _ints(mask, self.device, "mask", tokens, True), seqs, max_draft, scale,
            ws, nbytes))
        if rc:
            self._check(rc)

    def cache_free(self, cache, slots):
        """Release the pages of the given slots (int32 device tensor) and empty them."""
        rc = _lib.hyper_attn_cache_free(self._h, self._cache(cache), _ints(slots, self.device, "slots"), slots.numel())
        if rc:
            self._check(rc)

    def cache_fork(self, cache, src, dst):
        """Make the empty slots dst copies of the slots src; they share the pages of the committed rows."""
        n = src.numel()
        rc = _lib.hyper_attn_cache_fork(self._h, self._cache(cache), _ints(src, self.device, "src"),
                                        _ints(dst, self.device, "dst", n), n)
        if rc:
            self._check(rc)

    def cache_reserve(self, cache, slots, add, granted=None):
        """Room for add[i] more rows in slots[i]: new pages, and a copy of a shared last page. granted (int32, optional)
        gets add[i], or 0 where the free pages did not suffice."""
        n = slots.numel()
        L = _lib
        c = self._cache(cache)
        nbytes = L.hyper_attn_cache_workspace(n, cache.pages)
        ws = self._workspace(nbytes)
        rc = L.hyper_attn_cache_reserve(
            self._h, c, _ints(slots, self.device, "slots"), _ints(add, self.device, "add", n), n,
            None if granted is None else _ints(granted, self.device, "granted", n), ws, nbytes)
        if rc:
            self._check(rc)

    def cache_append(self, cache, slots, offsets, K, V, *, layer=0):
        """Write K, V [layers, tokens, kv_heads, d] to the cache's layers from `layer` on: rows offsets[i] ..
        offsets[i+1]-1 go behind the committed rows of slots[i] (reserved before)."""
        c = self._cache(cache)
        strides = []
        for t in (K, V):
            s = t.stride()
            if len(s) != 4 or (s[3] != 1 and t.shape[3] != 1) or t.dtype is not cache.dtype or t.get_device() != self.device:
                raise ValueError("K, V: [layers, tokens, kv_heads, d] of the cache's type on the handle's device, contiguous rows")
            strides.append(_APPEND.pack(s[0], s[1], s[2]))
        shape = K.shape
        if V.shape != shape or shape[2] != cache.kv_heads or shape[3] != cache.d:
            raise ValueError("K, V: the cache's kv_heads and d are needed")
        n = slots.numel()
        rc = _lib.hyper_attn_cache_append(
            self._h, c, _ints(slots, self.device, "slots"), _ints(offsets, self.device, "offsets", n + 1), n, shape[1],
            K.data_ptr(), V.data_ptr(), strides[0], strides[1], layer, shape[0])
        if rc:
            self._check(rc)

    def cache_commit(self, cache, slots, counts, keep=None):
        """Keep counts[i] of the rows behind the committed ones of slots[i]: the rows keep[i, :counts[i]] (ascending), or
        the first ones; they become committed, the pages behind them are released."""
        n = slots.numel()
        most = 0
        if keep is not None:
            kshape = keep.shape
            if len(kshape) != 2 or kshape[0] != n:
                raise ValueError("keep: [n, max_keep] is needed")
            most = kshape[1]
        rc = _lib.hyper_attn_cache_commit(
            self._h, self._cache(cache), _ints(slots, self.device, "slots"), _ints(counts, self.device, "counts", n),
            None if keep is None else _ints(keep, self.device, "keep"), most, n)
        if rc:
            self._check(rc)

    def debug_copy(self, what: str, level: int, dtype, count: int) -> np.ndarray:
        out = np.zeros(count, dtype)
        self._check(lib().hyper_attn_debug_copy(self._h, DBG[what], level, out.ctypes.data, out.nbytes))
        return out

    def status(self) -> int:
        return lib().hyper_attn_status(self._h)

    def last_error(self) -> str:
        return lib().hyper_attn_last_error(self._h).decode()

    def test_fail_alloc(self, count: int):
        """Test hook: fail the handle's next `count` allocations as if memory had run out (HA_ERR_OOM)."""
        self._check(lib().hyper_attn_test_fail_alloc(self._h, count))

    def profile(self, enable: bool):
        self._check(lib().hyper_attn_profile(self._h, int(enable)))

    def profile_read(self):
        """{class: (total ms, launches)} since the previous read (synchronises the stream)."""
        n = len(KERNEL_CLASSES)
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_int * n)()
        self._check(lib().hyper_attn_profile_read(self._h, ms, cnt, n))
        return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_CLASSES)}

    def last_kernel(self) -> str:
        """'simt' or 'tc': the attention kernel family of the last forward call."""
        return {0: "none", 1: "simt", 2: "tc"}[lib().hyper_attn_last_kernel(self._h)]

    def last_launch_count(self) -> int:
        return lib().hyper_attn_last_launch_count(self._h)

    def close(self):
        if self._h:
            lib().hyper_attn_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
