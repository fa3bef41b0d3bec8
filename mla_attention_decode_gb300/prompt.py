"""ctypes binding of include/mla_prompt.h: the attention of a prompt.

``MLAPrompt`` is the workspace of one batch layout; a call takes the query
projection's two parts, the up-projected keys and values, the position part of
the rows, and the documents' bounds.  As in ``mla_attention_decode_gb300.binding``
this marshals arguments only, nothing synchronises, and what only the device can
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
from .binding import MLA_OK, MLAError

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
        a = mla_prompt_args(num_q=self.num_tokens, num_kv=self.num_keys, batch=self.batch, heads=self.heads)
        nbytes = int(self._lib.mla_prompt_workspace_bytes(ctypes.addressof(a)))
        if nbytes == 0:
            raise MLAError(binding.MLA_ERR_INVALID_ARG, "mla_prompt_workspace_bytes")
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.device = self.workspace.device

    def _check(self, name, t, dtype, shape):
        if t.dtype != dtype or t.device != self.device or tuple(t.shape) != shape:
            raise ValueError(f"{name} is {dtype} {shape} on {self.device}: got {t.dtype} {tuple(t.shape)} on {t.device}")
        if t.dim() and t.numel() and t.stride(-1) != 1 and t.shape[-1] != 1:
            raise ValueError(f"{name}: the last dimension is consecutive")

    def __call__(self, q_nope, q_pe, k_nope, k_pe, v, qo_indptr, kv_indptr, prefix=None, out=None, lse=None, stream=None):
        """Attention of the query tokens over their documents' keys: (out [T, heads, 128] bf16, lse [T, heads]).

        ``q_nope`` [T, heads, 128], ``q_pe`` [T, heads, 64], ``k_nope`` and ``v`` [S, heads, 128], ``k_pe`` [S, 64]:
        bf16, any strides that are multiples of 8.  ``qo_indptr``, ``kv_indptr`` int32 [documents + 1]; ``prefix``
        int32 [documents]: that many keys are seen by every token.  Rows of no document are left as they were
        in ``out`` and ``lse`` (unset without them)."""
        t, s, b = q_nope.shape[0], k_nope.shape[0], qo_indptr.shape[0] - 1
        h, bf, i32 = self.heads, torch.bfloat16, torch.int32
        if t > self.num_tokens or s > self.num_keys or not 0 <= b <= self.batch:
            raise ValueError(f"made for {self.num_tokens} tokens, {self.num_keys} keys and {self.batch} documents: got {t}, {s}, {b}")
        for name, x, dtype, shape in (("q_nope", q_nope, bf, (t, h, NOPE)), ("q_pe", q_pe, bf, (t, h, PE)),
                                      ("k_nope", k_nope, bf, (s, h, NOPE)), ("k_pe", k_pe, bf, (s, PE)),
                                      ("v", v, bf, (s, h, V)), ("qo_indptr", qo_indptr, i32, (b + 1,)),
                                      ("kv_indptr", kv_indptr, i32, (b + 1,))):
            self._check(name, x, dtype, shape)
        if prefix is not None:
            self._check("prefix", prefix, i32, (b,))
        if out is None:
            out = torch.empty(t, h, V, dtype=bf, device=self.device)
        else:
            self._check("out", out, bf, (t, h, V))
        if lse is None:
            lse = torch.empty(t, h, dtype=torch.float32, device=self.device)
        else:
            self._check("lse", lse, torch.float32, (t, h))
            if not lse.is_contiguous():
                raise ValueError("lse is contiguous")
        a = mla_prompt_args(q_nope.data_ptr(), q_pe.data_ptr(), k_nope.data_ptr(), k_pe.data_ptr(), v.data_ptr(),
                            qo_indptr.data_ptr(), kv_indptr.data_ptr(), None if prefix is None else prefix.data_ptr(),
                            out.data_ptr(), lse.data_ptr(), q_nope.stride(0), q_nope.stride(1), q_pe.stride(0), q_pe.stride(1),
                            k_nope.stride(0), k_nope.stride(1), k_pe.stride(0), v.stride(0), v.stride(1), out.stride(0),
                            out.stride(1), t, s, b, h, self.causal, self.sm_scale)
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        with torch.cuda.device(self.device):
            rc = self._lib.mla_prompt_fwd(ctypes.addressof(a), self.workspace.data_ptr(), self.workspace.numel(), handle)
        if rc != MLA_OK:
            raise MLAError(rc, "mla_prompt_fwd")
        return out, lse

    def poll_error(self, stream=None) -> int:
        """The error that a call met on the device (0: none), cleared; synchronises the stream."""
        if stream is not None and not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=self.device)
        with torch.cuda.device(self.device):
            return binding.mla_decode_poll_error(self.workspace, stream)
