"""ctypes binding of include/mla_cache.h: the operators around the latent cache.

``MLACachePool`` is a paged cache with its pages' counts and a workspace; its
methods write rows (norms, rotation and storage format in one pass), read them
back as bf16, and manage the pages of a batch's sequences.  ``MLARope`` and
``MLANorm`` are the rotation and the norms of a layer.  As in
``mla_attention_decode_gb300.binding`` this marshals arguments only (compiled, in
``_mla_cache.so``, for the calls of a decode step): every step runs in the
library's CUDA kernels, nothing synchronises, and what only the device can see
is reported by ``MLACachePool.poll_error``.

A page table is a tuple ``(page_indptr, kv_indices, last_page_len)`` of int32
CUDA tensors, the arrays that ``PagedMLADecoder`` takes.  A decode step of one
token per sequence, with two tables used in turn:

    pool.resize(table, lengths, out=spare)                  # lengths: one more row each
    slots, rows = pool.slots(spare, qo_indptr, batch, rows=positions)
    for layer in ...:
        pool.append(kv_a[:, :512], kv_a[:, 512:], slots, rope, positions, norm,
                    q_pe=q_pe, q_out=q, layer=layer)        # q: latent columns there already
        decoder(q, pool.kv[layer], *spare, qo_indptr, kv_scale=...)   # a PagedMLADecoder for the lengths
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

from . import binding
from .binding import MLA_ERR_INVALID_ARG, MLA_KV_BF16, MLA_KV_FP8_E4M3, MLA_KV_MXFP4, MLA_OK, MLAError

MLA_ERR_OUT_OF_PAGES = 8
PAIRS = 32
ROW_WIDTH = {MLA_KV_BF16: 576, MLA_KV_FP8_E4M3: 576, MLA_KV_MXFP4: 288}
_PARTS = ("kv_lat", "kv_pe", "q_lat", "q_pe")
_PART_COLUMNS = (512, 64, 512, 64)


class mla_cache(ctypes.Structure):
    _fields_ = [("kv", ctypes.c_void_p), ("kv_scale", ctypes.c_void_p), ("kv_layer_bytes", ctypes.c_int64),
                ("scale_layer_bytes", ctypes.c_int64), ("kv_dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("num_layers", ctypes.c_int32), ("scale_stride", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("scale_width", ctypes.c_int32), ("reserved2", ctypes.c_int32)]


class mla_rope(ctypes.Structure):
    _fields_ = [("turn", ctypes.c_uint64 * PAIRS), ("axis", ctypes.c_uint8 * PAIRS), ("num_axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class mla_norm(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p * 4), ("apply", ctypes.c_int32), ("weight_fp32", ctypes.c_int32),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class mla_append_args(ctypes.Structure):
    _fields_ = [("kv_lat", ctypes.c_void_p), ("kv_pe", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("q_lat", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("kv_lat_stride", ctypes.c_int64), ("kv_pe_stride", ctypes.c_int64),
                ("position_stride", ctypes.c_int64), ("q_lat_token_stride", ctypes.c_int64),
                ("q_lat_head_stride", ctypes.c_int64), ("q_pe_token_stride", ctypes.c_int64),
                ("q_pe_head_stride", ctypes.c_int64), ("num_tokens", ctypes.c_int32), ("layer", ctypes.c_int32)]


class mla_page_table(ctypes.Structure):
    _fields_ = [("page_indptr", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p),
                ("last_page_len", ctypes.c_void_p), ("batch", ctypes.c_int32), ("num_indices", ctypes.c_int32)]


EXT_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_mla_cache.so")
EXT_TORCH_PATH = os.path.join(os.path.dirname(EXT_PATH), "_build", "ext_torch_version")
_ENTRY_POINTS = ("append", "gather", "slots", "copy_pages", "fork", "resize", "free", "compact")
_lock = threading.Lock()
_lib: ctypes.CDLL | None = None
_ext = None


def _load_extension():
    loader = importlib.machinery.ExtensionFileLoader("_mla_cache", EXT_PATH)
    ext = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_mla_cache", EXT_PATH, loader=loader))
    loader.exec_module(ext)
    return ext


def load_library() -> ctypes.CDLL:
    """The library with the entry points of mla_cache.h bound, and the extension that marshals
    their arguments; raises if either is missing."""
    global _lib, _ext
    if _lib is not None:
        return _lib
    lib = binding.load_library()
    with _lock:
        if _lib is None:
            P, i32, i64, sz, B = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_char_p
            for name, args in (("mla_rope_plan", [P, P, i32, i32, ctypes.c_double, P]),
                               ("mla_cache_append", [P, P, P, B, P, P]),
                               ("mla_cache_gather", [P, i32, P, i32, P, i64, P, P]),
                               ("mla_cache_slots", [P, B, P, i32, P, P, i64, P, P]),
                               ("mla_cache_copy_pages", [P, P, P, i32, P, P]),
                               ("mla_cache_fork", [P, P, B, P, B, P, sz, P]),
                               ("mla_cache_resize", [P, P, B, P, B, P, sz, P]),
                               ("mla_cache_free", [P, P, P, i32, P, P]),
                               ("mla_cache_compact", [P, P, P, P, P, i32, P, P, sz, P])):
                getattr(lib, name).argtypes = args
                getattr(lib, name).restype = ctypes.c_int
            lib.mla_cache_workspace_bytes.argtypes = [P, i32]
            lib.mla_cache_workspace_bytes.restype = sz
            if not os.path.exists(EXT_PATH):
                raise RuntimeError(f"{EXT_PATH} is missing: build it with `python -m mla_attention_decode_gb300.build`")
            this = str(torch.__version__)
            built_for = open(EXT_TORCH_PATH).read() if os.path.exists(EXT_TORCH_PATH) else this
            if built_for == this:  # (else it may not even load)
                ext = _load_extension()
                built_for = ext.torch_version
            if built_for != this:
                raise RuntimeError(f"{EXT_PATH} was built for torch {built_for}, this is {this}: build it again")
            ext.bind(*(ctypes.cast(getattr(lib, "mla_cache_" + n), ctypes.c_void_p).value for n in _ENTRY_POINTS))
            _ext, _lib = ext, lib
    return _lib


class MLARope:
    """The rotation of the 64 position columns (32 pairs).

    ``inv_freq``: 32 angles per position step (default ``theta ** (-i / 32)``);
    ``axis_of_pair``: which of a token's positions turns each pair (default: all
    the first), or ``sections``: that many pairs for each axis in turn;
    ``interleaved``: pair i is columns (2i, 2i + 1), else (i, i + 32); ``scale``:
    a factor on the rotated columns."""

    def __init__(self, inv_freq=None, axis_of_pair=None, sections=None, interleaved: bool = True, scale: float = 1.0,
                 theta: float = 10000.0):
        freq = [float(theta) ** (-i / PAIRS) for i in range(PAIRS)] if inv_freq is None else [float(f) for f in inv_freq]
        if sections is not None:
            if axis_of_pair is not None:
                raise ValueError("give axis_of_pair or sections, not both")
            axis_of_pair = [a for a, n in enumerate(sections) for _ in range(int(n))]
        axes = [0] * PAIRS if axis_of_pair is None else [int(a) for a in axis_of_pair]
        if len(freq) != PAIRS or len(axes) != PAIRS:
            raise ValueError(f"a rotation has {PAIRS} pairs: got {len(freq)} frequencies and {len(axes)} axes")
        self.num_axes = max(axes) + 1
        self.rope = mla_rope()
        rc = load_library().mla_rope_plan((ctypes.c_double * PAIRS)(*freq), (ctypes.c_int32 * PAIRS)(*axes),
                                          self.num_axes, int(bool(interleaved)), float(scale),
                                          ctypes.addressof(self.rope))
        if rc != MLA_OK:
            raise MLAError(rc, "mla_rope_plan")
        self.address = ctypes.addressof(self.rope)


class MLANorm:
    """Root-mean-square norms of a key row's and of each query head's parts.

    ``kv_lat``, ``kv_pe``, ``q_lat``, ``q_pe``: the weights of the part (a CUDA
    tensor of 512 or 64, bf16 or fp32, one type for all), True for weights of 1,
    or None where the part is not normed."""

    def __init__(self, eps: float = 1e-6, kv_lat=None, kv_pe=None, q_lat=None, q_pe=None):
        self.norm = mla_norm(eps=float(eps))
        self.weights = []  # kept alive
        self.device = None
        dtypes = set()
        for i, w in enumerate((kv_lat, kv_pe, q_lat, q_pe)):
            if w is None or w is False:
                continue
            self.norm.apply |= 1 << i
            if w is True:
                continue
            if w.numel() != _PART_COLUMNS[i] or not w.is_contiguous() or not w.is_cuda:
                raise ValueError(f"{_PARTS[i]}: the weights are a contiguous CUDA tensor of {_PART_COLUMNS[i]}")
            if w.dtype not in (torch.bfloat16, torch.float32):
                raise ValueError(f"{_PARTS[i]}: the weights are bf16 or fp32, not {w.dtype}")
            if self.device is not None and w.device != self.device:
                raise ValueError("the weights are on different devices")
            dtypes.add(w.dtype)
            self.device = w.device
            self.weights.append(w)
            self.norm.weight[i] = w.data_ptr()
        if len(dtypes) > 1:
            raise ValueError("the weights are all bf16 or all fp32")
        self.norm.weight_fp32 = int(torch.float32 in dtypes)
        self.device_index = -1 if self.device is None else self.device.index
        self.address = ctypes.addressof(self.norm)


class MLACachePool:
    """A paged latent cache: its rows, the counts of its pages and a workspace.

    ``kv``: [rows, width] or [layers, rows, width] (rows = pages * page_size):
    bf16 [.., 576], e4m3 bytes [.., 576] or packed e2m1 [.., 288]; ``kv_scale``:
    fp32 [1] (or one per layer) for fp8, e8m0 bytes [(layers,) rows, >= 18] for
    MXFP4 (columns of a wider tensor too, 16-byte aligned: the others are left
    alone).  ``refs``: int32, how many sequences hold each page (default: all
    free; a table made elsewhere has its pages counted here before ``fork`` or
    ``resize`` take it: a page that nobody holds is no page of a sequence).  A
    contiguous cache is one with pages of one row.

    Calls that share a pool are ordered on the GPU (one stream, or events).
    Methods enqueue on ``stream`` (default: torch's current one) of the pool's
    device; ``poll_error`` synchronises.  As with any kernel, memory that a call
    on another stream uses is the caller's to keep (``Tensor.record_stream``)."""

    def __init__(self, kv, kv_dtype, page_size: int, kv_scale=None, refs=None, max_batch: int = 4096):
        self.kv_dtype = binding._dtype_code(kv_dtype)
        if self.kv_dtype not in ROW_WIDTH:
            raise MLAError(binding.MLA_ERR_UNSUPPORTED, "MLACachePool")
        if kv.dim() not in (2, 3):
            raise ValueError("kv is [rows, width] or [layers, rows, width]")
        if not kv.is_cuda:
            raise ValueError("kv is a CUDA tensor")
        layered = kv.dim() == 3
        width, want = ROW_WIDTH[self.kv_dtype], (torch.bfloat16,)
        if self.kv_dtype != MLA_KV_BF16:
            want = (torch.uint8, torch.float8_e4m3fn) if self.kv_dtype == MLA_KV_FP8_E4M3 else (torch.uint8,)
        if kv.dtype not in want or kv.shape[-1] != width or kv.stride(-1) != 1 or kv.stride(-2) != width:
            raise ValueError(f"kv is {want[0]} [.., {width}] with consecutive rows: got {kv.dtype} {tuple(kv.shape)}")
        page_size, rows = int(page_size), kv.shape[-2]
        if page_size < 1 or rows % page_size:
            raise ValueError(f"{rows} rows are not whole pages of {page_size}")
        c = self.cache = mla_cache(kv=kv.data_ptr(), kv_dtype=self.kv_dtype, page_size=page_size,
                                   num_pages=rows // page_size, num_layers=kv.shape[0] if layered else 1)
        if layered and kv.shape[0] > 1:
            c.kv_layer_bytes = kv.stride(0) * kv.element_size()
        if self.kv_dtype == MLA_KV_BF16:
            if kv_scale is not None:
                raise ValueError("a bf16 cache has no scales")
        else:
            if kv_scale is None or kv_scale.device != kv.device:
                raise ValueError("kv_scale is on the cache's device")
            if self.kv_dtype == MLA_KV_FP8_E4M3:
                if kv_scale.dtype != torch.float32 or kv_scale.numel() not in (1, c.num_layers) or not kv_scale.is_contiguous():
                    raise ValueError("kv_scale is fp32, one or one per layer")
                c.scale_layer_bytes = 4 if kv_scale.numel() > 1 else 0
            else:
                if (kv_scale.dtype != torch.uint8 or kv_scale.shape[:-1] != kv.shape[:-1] or kv_scale.shape[-1] < 18
                        or kv_scale.stride(-1) != 1):
                    raise ValueError("kv_scale is uint8 [.., rows, >= 18]")
                # the columns of a wider tensor: what lies between them is not the cache's.  (One row has no
                # stride that means anything.)
                c.scale_stride = kv_scale.stride(-2) if rows > 1 else kv_scale.shape[-1]
                if kv_scale.shape[-1] < c.scale_stride:
                    c.scale_width = kv_scale.shape[-1]
                if layered and kv.shape[0] > 1:
                    c.scale_layer_bytes = kv_scale.stride(0)
            c.kv_scale = kv_scale.data_ptr()
        self.kv, self.kv_scale, self.device = kv, kv_scale, kv.device
        self.page_size, self.num_pages, self.num_layers = page_size, c.num_pages, c.num_layers
        if refs is None:
            refs = torch.zeros(self.num_pages, dtype=torch.int32, device=self.device)
        if refs.dtype != torch.int32 or refs.device != self.device or refs.shape != (self.num_pages,):
            raise ValueError(f"refs is int32 [{self.num_pages}] on {self.device}")
        self.refs = refs
        lib = load_library()
        nbytes = int(lib.mla_cache_workspace_bytes(ctypes.addressof(c), int(max_batch)))
        if nbytes == 0:
            raise MLAError(MLA_ERR_INVALID_ARG, "mla_cache_workspace_bytes")
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self._core = _ext.core(ctypes.addressof(c), self.workspace.data_ptr(), nbytes, self.device.index)

    @classmethod
    def allocate(cls, kv_dtype, num_pages: int, page_size: int, num_layers: int = 1, device="cuda", kv_scale=1.0,
                 max_batch: int = 4096):
        """A pool over new, zeroed storage; ``kv_scale``: fp8 only, the scale of every layer."""
        code, rows = binding._dtype_code(kv_dtype), int(num_pages) * int(page_size)
        kv = torch.zeros(num_layers, rows, ROW_WIDTH[code], device=device,
                         dtype=torch.bfloat16 if code == MLA_KV_BF16 else torch.uint8)
        scale = None
        if code == MLA_KV_FP8_E4M3:
            scale = torch.full((1,), float(kv_scale), dtype=torch.float32, device=device)
        elif code == MLA_KV_MXFP4:
            # layers 16-byte aligned, as the decode takes them: whole runs of 8 rows
            scale = torch.full((num_layers, -(-rows // 8) * 8, 18), 127, dtype=torch.uint8, device=device)[:, :rows]
        return cls(kv, code, page_size, kv_scale=scale, max_batch=max_batch)

    def table(self, batch: int, num_indices: int):
        """Buffers of a page table of ``batch`` empty sequences, with room for ``num_indices`` entries (all -1)."""
        return (torch.zeros(batch + 1, dtype=torch.int32, device=self.device),
                torch.full((num_indices,), -1, dtype=torch.int32, device=self.device),
                torch.zeros(batch, dtype=torch.int32, device=self.device))

    # -------------------------------------------------------------- rows
    def append(self, kv_lat, kv_pe, slots, rope: MLARope | None = None, positions=None, norm: MLANorm | None = None,
               q_pe=None, q_lat=None, q_out=None, layer: int = 0, stream=None):
        """Norms, rotates and stores T tokens' key rows; norms and rotates their queries into ``q_out``.

        ``kv_lat`` [T, 512], ``kv_pe`` [T, 64] (with ``slots`` None, None, None: queries only), ``slots`` [T] (-1: not
        stored), ``positions`` [T] or [T, axes], ``q_pe`` [T, 16, 64], ``q_lat`` [T, 16, 512] (None: the latent columns
        of ``q_out`` stay), ``q_out`` [T, 16, 576] contiguous; bf16, the last dimension consecutive."""
        rc = _ext.append(self._core, kv_lat, kv_pe, slots, rope, positions, norm, q_pe, q_lat, q_out, layer, stream)
        if rc:
            raise MLAError(rc, "mla_cache_append")

    def gather(self, slots, out=None, layer: int = 0, stream=None):
        """Rows ``slots`` of a layer as bf16 [T, 576] (``out``'s rows with slot -1 stay as they were; without
        ``out`` they are unset)."""
        rc, out = _ext.gather(self._core, slots, out, layer, stream)
        if rc:
            raise MLAError(rc, "mla_cache_gather")
        return out

    def slots(self, table, qo_indptr, num_tokens: int, slots=None, rows=None, stream=None):
        """The cache row of each sequence's last ``qo_indptr[b + 1] - qo_indptr[b]`` tokens, as ``slots`` [num_tokens]
        (-1 past the batch); with ``rows`` (int32, any stride) the tokens' places in their sequences too."""
        rc, slots = _ext.slots(self._core, table, qo_indptr, num_tokens, slots, rows, stream)
        if rc:
            raise MLAError(rc, "mla_cache_slots")
        return slots, rows

    # -------------------------------------------------------------- pages
    @property
    def refs(self):
        """How many sequences hold each page, int32 [pages].  Assigning another tensor makes its counts the pool's."""
        return self._refs

    @refs.setter
    def refs(self, refs):
        self._refs, self._left = refs, None

    def _settle(self):
        """Before counts change that a compaction has left by the old numbers."""
        if self._left == self._refs._version:
            raise ValueError("compact(out=...) has left the pool's counts by the old page numbers: make the new counts "
                             "the pool's (pool.refs = refs), or keep the old table (pool.refs = pool.refs)")
        self._left = None  # they have been written since

    def copy_pages(self, src, dst, stream=None):
        """Page ``dst[i]`` becomes a copy of page ``src[i]``, in every layer."""
        rc = _ext.copy_pages(self._core, src, dst, stream)
        if rc:
            raise MLAError(rc, "mla_cache_copy_pages")

    def fork(self, table, parents, out, stream=None):
        """Writes to ``out`` a batch whose sequence n is a fork of ``table``'s sequence ``parents[n]``."""
        if self._left is not None:
            self._settle()
        rc = _ext.fork(self._core, self._refs, table, parents, out, stream)
        if rc:
            raise MLAError(rc, "mla_cache_fork")
        return out

    def resize(self, table, lengths, out, stream=None):
        """Writes to ``out`` the table whose sequence b has ``lengths[b]`` rows; ``table`` is void from then on.
        Lengths of 0 end a batch, or some of its sequences: what they hold is given back, however long they are."""
        if self._left is not None:
            self._settle()
        rc = _ext.resize(self._core, self._refs, table, lengths, out, stream)
        if rc:
            raise MLAError(rc, "mla_cache_resize")
        return out

    def free(self, pages, stream=None):
        """Ends one hold on each of ``pages`` (-1 is skipped): of a table, the entries that are in use, and only those.
        What lies behind them in a buffer that was used before are pages too, and holds of others may end; where the
        host does not know how many are in use, ``resize`` to lengths of 0 ends them."""
        if self._left is not None:
            self._settle()
        rc = _ext.free(self._core, self._refs, pages, stream)
        if rc:
            raise MLAError(rc, "mla_cache_free")

    def compact(self, kv_indices, out=None, stream=None):
        """Moves the pages in use to the front and renumbers ``kv_indices`` (the entries of a table that are in use).
        ``out``: (kv_indices, refs, live [1]) to write; without it the pool's counts are rewritten in place and the
        other two are new.  Returns the three.

        Counts written to a tensor of ``out``'s own leave the pool's as they were, by the old numbers (which still
        hold for the old table: the pages moved from keep their rows).  ``fork``, ``resize`` and ``free`` refuse from
        then on until it is said which counts go on: ``pool.refs = refs`` with the new table (or the new counts copied
        into ``pool.refs``), ``pool.refs = pool.refs`` with the old one.  (Inference tensors do not tell whether they
        have been written: over such counts nothing is refused.)"""
        indices, refs, live = (None, None, None) if out is None else out
        rc, indices, refs, live = _ext.compact(self._core, self._refs, kv_indices, indices, refs, live, stream)
        if rc:
            raise MLAError(rc, "mla_cache_compact")
        own = self._refs
        apart = refs is not own and refs.data_ptr() != own.data_ptr() and not own.is_inference()
        self._left = own._version if apart else None
        return indices, refs, live

    def poll_error(self, stream=None) -> int:
        """The error that a call on this pool met on the device (0: none), cleared; synchronises the stream."""
        if stream is not None and not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=self.device)
        with torch.cuda.device(self.device):
            return binding.mla_decode_poll_error(self.workspace, stream)
