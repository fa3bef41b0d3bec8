"""ctypes binding of include/mla_prompt.h: the attention of a prompt.

``MLAPrompt`` is the workspace of one batch layout; a call takes the query
projection's two parts, the up-projected keys and values, the position part of
the rows, and the documents' bounds.  As in ``mla_attention_decode_gb300.cache``
this marshals arguments only (compiled), nothing synchronises, and what only the device can
see is reported by ``poll_error``.

The next chunk of a prompt whose context is cached:

    pool.append(kv_a[:, :512], kv_a[:, 512:], slots, rope, positions, norm, q_pe=q_b[..., 128:], q_out=q)
    rows = pool.gather(context_slots)                                  # the chunk's own among them
    kv_b = (rows[:, :512] @ w_kv_b).view(-1, heads, 256)
    out, lse = prompt(q_b[..., :128], q[..., 512:], kv_b[..., :128], rows[:, 512:], kv_b[..., 128:],
                      qo_indptr, kv_indptr)
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import binding
from .binding import MLAError
from .cache import extension

NOPE, PE, V = 128, 64, 128
_STRIDES = ("q_nope_token_stride", "q_nope_head_stride", "q_pe_token_stride", "q_pe_head_stride", "k_nope_token_stride",
            "k_nope_head_stride", "k_pe_token_stride", "v_token_stride", "v_head_stride", "out_token_stride",
            "out_head_stride")


class mla_prompt_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q_nope", "q_pe", "k_nope", "k_pe", "v", "qo_indptr", "kv_indptr",
                                                "prefix", "out", "lse")] +
                [(n, ctypes.c_int64) for n in _STRIDES] +
                [(n, ctypes.c_int32) for n in ("num_q", "num_kv", "batch", "heads", "causal")] +
                [("sm_scale", ctypes.c_float)])


def load_library() -> ctypes.CDLL:
    """The library with the entry points of mla_prompt.h bound."""
    lib = binding.load_library()
    if lib.mla_prompt_fwd.argtypes is None:
        P, sz = ctypes.c_void_p, ctypes.c_size_t
        lib.mla_prompt_workspace_bytes.argtypes, lib.mla_prompt_workspace_bytes.restype = [P], sz
        lib.mla_prompt_fwd.argtypes, lib.mla_prompt_fwd.restype = [P, P, sz, P], ctypes.c_int
    return lib


class MLAPrompt:
    """Workspace for prompts of up to ``num_tokens`` query tokens and ``num_keys`` keys in ``batch`` documents.

    ``causal``: token i of a document sees the keys up to its own (the document's last
    keys are its tokens'), else all of the document's.  ``sm_scale``: default
    1 / sqrt(192).  Calls that share an object are ordered on the GPU."""

    def __init__(self, num_tokens: int, num_keys: int, batch: int, heads: int = 16, causal: bool = True,
                 sm_scale: float = 1 / math.sqrt(NOPE + PE), device="cuda"):
        self.num_tokens, self.num_keys, self.batch, self.heads = int(num_tokens), int(num_keys), int(batch), int(heads)
        self.causal, self.sm_scale = bool(causal), float(sm_scale)
        self._lib = load_library()
        if max(map(abs, (self.num_tokens, self.num_keys, self.batch, self.heads))) >= 1 << 31:  # (a ctypes field would wrap)
            raise MLAError(binding.MLA_ERR_INVALID_ARG, "mla_prompt_workspace_bytes")
        a = mla_prompt_args(num_q=self.num_tokens, num_kv=self.num_keys, batch=self.batch, heads=self.heads)
        nbytes = int(self._lib.mla_prompt_workspace_bytes(ctypes.addressof(a)))
        if nbytes == 0:
            raise MLAError(binding.MLA_ERR_INVALID_ARG, "mla_prompt_workspace_bytes")
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.device = self.workspace.device
        if not self.workspace.is_cuda:
            raise ValueError("a prompt runs on a CUDA device")
        self._ext = extension()
        self._core = self._ext.prompt_core(self.workspace.data_ptr(), nbytes, self.device.index, self.num_tokens, self.num_keys,
                                           self.batch, self.heads, int(self.causal), self.sm_scale)

    def __call__(self, q_nope, q_pe, k_nope, k_pe, v, qo_indptr, kv_indptr, prefix=None, out=None, lse=None, stream=None):
        """Attention of the query tokens over their documents' keys: (out [T, heads, 128] bf16, lse [T, heads]).

        ``q_nope`` [T, heads, 128], ``q_pe`` [T, heads, 64], ``k_nope`` and ``v`` [S, heads, 128], ``k_pe`` [S, 64]:
        bf16, any strides that are multiples of 8.  ``qo_indptr``, ``kv_indptr`` int32 [documents + 1]; ``prefix``
        int32 [documents]: that many keys are seen by every token.  Rows of no document are left as they were
        in ``out`` and ``lse`` (unset without them)."""
        rc, out, lse = self._ext.prompt(self._core, q_nope, q_pe, k_nope, k_pe, v, qo_indptr, kv_indptr, prefix, out, lse, stream)
        if rc:
            raise MLAError(rc, "mla_prompt_fwd")
        return out, lse

    def poll_error(self, stream=None) -> int:
        """The error that a call met on the device (0: none), cleared; synchronises the stream."""
        if stream is not None and not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=self.device)
        with torch.cuda.device(self.device):
            return binding.mla_decode_poll_error(self.workspace, stream)
