"""Python binding of libgdnreplay (ReplaySSM verify / accept / flush of Gated
DeltaNet state on sm_103a).

Argument marshalling only: every step of the path runs in the CUDA kernels of
``csrc/`` behind the C ABI declared in ``include/`` (``gdnreplay.h``: the recurrence;
``gdnlayer.h``, ``gdnattn.h``, ``gdndraft.h``: what stands beside it).
PyTorch supplies device memory and the current stream.  There is no CPU
fallback: if the shared library cannot be built or loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

__all__ = ["Dims", "GdnError", "load", "gdn_replay_verify", "gdn_replay_accept",
           "gdn_replay_flush", "gdn_replay_verify_fold", "gdn_replay_accept_fold",
           "gdn_replay_kernel_family", "gdn_replay_strerror", "STATUS_BAD_ACCEPT",
           "STATUS_NO_ROOM", "STATUS_BAD_LEN", "STATUS_BAD_SLOT", "STATUS_TIMEOUT",
           "STATUS_DRAIN", "FLAG_TEST_EXPIRE", "FLAG_TWO_TERMS", "FAMILY_TCGEN05", "FAMILY_PERTOKEN", "DTYPE_BF16",
           "DTYPE_F32", "ReplayLayer", "ConvDims", "gdn_conv_verify", "gdn_conv_accept",
           "gdn_gated_rmsnorm_fp8", "ConvLayer", "CONV_ACT_NONE", "CONV_ACT_SILU",
           "gdn_nonreplay_verify", "gdn_nonreplay_accept", "NonReplayLayer",
           "PageDims", "AttnDims", "RopeDims", "PagedCache", "AttnLayer", "ROPE_HALF", "ROPE_PAIRS",
           "STATUS_BAD_PAGE", "STATUS_BAD_POS", "STATUS_BAD_TREE", "STATUS_NO_PAGES", "AdvanceDims",
           "gdn_replay_advance", "gdn_replay_advance_workspace", "gdn_conv_advance", "DraftDims", "DraftSampler",
           "STATUS_BAD_TOKEN", "STATUS_BAD_PROB"]

DTYPE_BF16, DTYPE_F32 = 0, 1
STATUS_BAD_ACCEPT, STATUS_NO_ROOM, STATUS_BAD_LEN, STATUS_BAD_SLOT, STATUS_TIMEOUT = 1, 2, 4, 8, 16
STATUS_DRAIN = 32
STATUS_BAD_PAGE, STATUS_BAD_POS, STATUS_BAD_TREE, STATUS_NO_PAGES = 64, 128, 256, 512
STATUS_BAD_TOKEN, STATUS_BAD_PROB = 1024, 2048
FLAG_TEST_EXPIRE = 1
FLAG_TWO_TERMS = 4                   # AttnDims: AttnLayer.chunk in bf16 keeps two terms of a softmax weight
FAMILY_TCGEN05, FAMILY_PERTOKEN = 1, 2
FAMILY_NAMES = {FAMILY_TCGEN05: "tcgen05", FAMILY_PERTOKEN: "per-token"}
CONV_ACT_NONE, CONV_ACT_SILU = 0, 1
ROPE_HALF, ROPE_PAIRS = 0, 1
_TORCH_IN = {DTYPE_BF16: torch.bfloat16, DTYPE_F32: torch.float32}


class Dims(ctypes.Structure):
    """Mirror of ``gdn_replay_dims``."""
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("dk", ctypes.c_int32),
                ("dv", ctypes.c_int32), ("T", ctypes.c_int32), ("cap", ctypes.c_int32),
                ("threshold", ctypes.c_int32), ("n_slot", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("flags", ctypes.c_int32)]

    def __repr__(self):
        return "Dims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class AdvanceDims(ctypes.Structure):
    """Mirror of ``gdn_advance_dims``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "H", "Hk", "dk", "dv", "n_slot", "in_dtype")] + \
               [("scale", ctypes.c_float), ("flags", ctypes.c_int32)] + \
               [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")]

    def __repr__(self):
        return "AdvanceDims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class DraftDims(ctypes.Structure):
    """Mirror of ``gdn_draft_dims`` (include/gdndraft.h); the strides are taken from each call's tensors."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "V", "flags")] + \
               [(n, ctypes.c_int64) for n in ("p_stride", "q_stride")]

    def __repr__(self):
        return "DraftDims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class ConvDims(ctypes.Structure):
    """Mirror of ``gdn_conv_dims`` (include/gdnlayer.h)."""
    _fields_ = [("B", ctypes.c_int32), ("D", ctypes.c_int32), ("W", ctypes.c_int32),
                ("T", ctypes.c_int32), ("cap", ctypes.c_int32), ("n_slot", ctypes.c_int32),
                ("act", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]

    def __repr__(self):
        return "ConvDims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class PageDims(ctypes.Structure):
    """Mirror of ``gdn_page_cache`` (include/gdnattn.h); the pointers are PagedCache's."""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("n_slot", "max_pages", "n_page", "page", "n_layer", "Hkv", "d", "dtype")] + \
               [(n, ctypes.c_void_p) for n in
                ("k", "v", "block_table", "seq_len", "n_owned", "ref", "free_list", "free_count")]

    def __repr__(self):
        return "PageDims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_[:8]) + ")"


class AttnDims(ctypes.Structure):
    """Mirror of ``gdn_attn_dims``."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("scale", ctypes.c_float), ("flags", ctypes.c_int32)]

    def __repr__(self):
        return "AttnDims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class RopeDims(ctypes.Structure):
    """Mirror of ``gdn_rope_dims``; the strides are taken from each call's tensors."""
    _fields_ = [("rot", ctypes.c_int32), ("style", ctypes.c_int32), ("max_pos", ctypes.c_int32),
                ("eps", ctypes.c_float), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]

    def __repr__(self):
        return "RopeDims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class GdnError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {code} ({gdn_replay_strerror(code)})")
        self.code = code


_lib = None


def load(rebuild: bool = False) -> ctypes.CDLL:
    """Build (if stale) and load libgdnreplay.so; raises if that is impossible."""
    global _lib
    if _lib is None or rebuild:
        path = _build.build(force=rebuild)
        if not os.path.exists(path):
            raise RuntimeError(f"libgdnreplay not found at {path}")
        lib = ctypes.CDLL(path)
        P, I = ctypes.c_void_p, ctypes.c_int32
        D = ctypes.POINTER(Dims)
        lib.gdn_replay_verify.argtypes = [D] + [P] * 15
        lib.gdn_replay_accept.argtypes = [D, P, P, P, P, P]
        lib.gdn_replay_flush.argtypes = [D] + [P] * 7 + [I, P, P]
        lib.gdn_replay_verify_fold.argtypes = [D] + [P] * 15
        lib.gdn_replay_accept_fold.argtypes = [D, P, P, P, P, P]
        lib.gdn_replay_strerror.argtypes = [ctypes.c_int]
        lib.gdn_replay_strerror.restype = ctypes.c_char_p
        lib.gdn_replay_version.argtypes = []
        lib.gdn_replay_kernel_family.argtypes = [D]
        CD = ctypes.POINTER(ConvDims)
        lib.gdn_conv_verify.argtypes = [CD] + [P] * 9
        lib.gdn_conv_accept.argtypes = [CD, P, P, P, P, P]
        lib.gdn_gated_rmsnorm_fp8.argtypes = [I, I, P, P, I, P, ctypes.c_float, ctypes.c_float, P, P]
        lib.gdn_nonreplay_verify.argtypes = [D] + [P] * 11
        lib.gdn_nonreplay_accept.argtypes = [D] + [P] * 6
        C, A, R = ctypes.POINTER(PageDims), ctypes.POINTER(AttnDims), ctypes.POINTER(RopeDims)
        lib.gdn_attn_stage.argtypes = [C, I, A, R] + [P] * 12
        lib.gdn_tree_build.argtypes = [C, A] + [P] * 7
        lib.gdn_attn_verify.argtypes = [C, I, A] + [P] * 7 + [ctypes.c_int64, P, P]
        lib.gdn_attn_workspace.argtypes = [C, A]
        lib.gdn_attn_workspace.restype = ctypes.c_int64
        lib.gdn_attn_accept.argtypes = [C, I, I] + [P] * 6
        lib.gdn_pages_reserve.argtypes = [C, I, P, I, P, P]
        lib.gdn_pages_fork.argtypes = [C, I] + [P] * 5
        lib.gdn_pages_copy.argtypes = [C, I] + [P] * 3
        lib.gdn_pages_release.argtypes = [C, I] + [P] * 3
        AD, DD = ctypes.POINTER(AdvanceDims), ctypes.POINTER(DraftDims)
        lib.gdn_replay_advance.argtypes = [AD] + [P] * 12 + [ctypes.c_int64, P, P]
        lib.gdn_replay_advance_workspace.argtypes = [AD]
        lib.gdn_replay_advance_workspace.restype = ctypes.c_int64
        lib.gdn_conv_advance.argtypes = [CD] + [P] * 11
        lib.gdn_attn_chunk.argtypes = [C, I, A] + [P] * 6 + [ctypes.c_int64, P, P]
        lib.gdn_attn_chunk_workspace.argtypes = [C, A]
        lib.gdn_attn_chunk_workspace.restype = ctypes.c_int64
        lib.gdn_draft_accept.argtypes = [DD] + [P] * 11
        for f in (lib.gdn_replay_advance, lib.gdn_conv_advance, lib.gdn_attn_chunk, lib.gdn_draft_accept):
            f.restype = ctypes.c_int
        for f in (lib.gdn_attn_stage, lib.gdn_tree_build, lib.gdn_attn_verify, lib.gdn_attn_accept,
                  lib.gdn_pages_reserve, lib.gdn_pages_fork, lib.gdn_pages_copy, lib.gdn_pages_release):
            f.restype = ctypes.c_int
        for f in (lib.gdn_conv_verify, lib.gdn_conv_accept, lib.gdn_gated_rmsnorm_fp8,
                  lib.gdn_nonreplay_verify, lib.gdn_nonreplay_accept):
            f.restype = ctypes.c_int
        for f in (lib.gdn_replay_verify, lib.gdn_replay_accept, lib.gdn_replay_flush,
                  lib.gdn_replay_verify_fold, lib.gdn_replay_accept_fold, lib.gdn_replay_version,
                  lib.gdn_replay_kernel_family):
            f.restype = ctypes.c_int
        _lib = lib
    return _lib


def gdn_replay_strerror(code: int) -> str:
    return load().gdn_replay_strerror(int(code)).decode()


def gdn_replay_kernel_family(d: Dims) -> int:
    """FAMILY_TCGEN05 or FAMILY_PERTOKEN: the kernels calls with dims d launch."""
    rc = load().gdn_replay_kernel_family(ctypes.byref(d))
    _check("gdn_replay_kernel_family", rc if rc < 0 else 0)
    return rc


def _sizes(d: Dims) -> dict:
    """Elements of each argument for dims d (the dense layouts of gdnreplay.h)."""
    B, H, dk, dv, T, cap, n = d.B, d.H, d.dk, d.dv, d.T, d.cap, d.n_slot
    return {"state": n * H * dv * dk, "state_idx": B, "buf_k": n * H * cap * dk,
            "buf_v": n * H * cap * dv, "buf_g": n * H * cap, "buf_beta": n * H * cap,
            "buf_len": n, "q": B * T * H * dk, "k": B * T * H * dk, "v": B * T * H * dv,
            "g": B * T * H, "beta": B * T * H, "out": B * T * H * dv, "accepted": B, "status": 1}


def _check_sizes(d: Dims, **tensors):
    """Every tensor must hold at least what the kernels read or write for dims d."""
    need = _sizes(d)
    for name, t in tensors.items():
        if isinstance(t, torch.Tensor) and t.numel() < need[name]:
            raise ValueError(f"{name}: needs at least {need[name]} elements for {d}, got {t.numel()}")


def _ptr(t, dtype=None, name=""):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise GdnError(fn, rc)


def gdn_replay_verify(d: Dims, state, state_idx, buf_k, buf_v, buf_g, buf_beta, buf_len,
                      q, k, v, g, beta, out, status, stream=None):
    tin = _TORCH_IN.get(d.in_dtype)
    f32, i32 = torch.float32, torch.int32
    _check_sizes(d, state=state, state_idx=state_idx, buf_k=buf_k, buf_v=buf_v, buf_g=buf_g,
                 buf_beta=buf_beta, buf_len=buf_len, q=q, k=k, v=v, g=g, beta=beta, out=out,
                 status=status)
    rc = load().gdn_replay_verify(
        ctypes.byref(d), _ptr(state, f32, "state"), _ptr(state_idx, i32, "state_idx"),
        _ptr(buf_k, tin, "buf_k"), _ptr(buf_v, tin, "buf_v"), _ptr(buf_g, f32, "buf_g"),
        _ptr(buf_beta, f32, "buf_beta"), _ptr(buf_len, i32, "buf_len"),
        _ptr(q, tin, "q"), _ptr(k, tin, "k"), _ptr(v, tin, "v"), _ptr(g, f32, "g"),
        _ptr(beta, f32, "beta"), _ptr(out, f32, "out"), _ptr(status, i32, "status"),
        _stream(stream))
    _check("gdn_replay_verify", rc)


def gdn_replay_verify_fold(d: Dims, state, state_idx, buf_k, buf_v, buf_g, buf_beta, buf_len,
                           q, k, v, g, beta, out, status, stream=None):
    tin = _TORCH_IN.get(d.in_dtype)
    f32, i32 = torch.float32, torch.int32
    _check_sizes(d, state=state, state_idx=state_idx, buf_k=buf_k, buf_v=buf_v, buf_g=buf_g,
                 buf_beta=buf_beta, buf_len=buf_len, q=q, k=k, v=v, g=g, beta=beta, out=out,
                 status=status)
    rc = load().gdn_replay_verify_fold(
        ctypes.byref(d), _ptr(state, f32, "state"), _ptr(state_idx, i32, "state_idx"),
        _ptr(buf_k, tin, "buf_k"), _ptr(buf_v, tin, "buf_v"), _ptr(buf_g, f32, "buf_g"),
        _ptr(buf_beta, f32, "buf_beta"), _ptr(buf_len, i32, "buf_len"),
        _ptr(q, tin, "q"), _ptr(k, tin, "k"), _ptr(v, tin, "v"), _ptr(g, f32, "g"),
        _ptr(beta, f32, "beta"), _ptr(out, f32, "out"), _ptr(status, i32, "status"),
        _stream(stream))
    _check("gdn_replay_verify_fold", rc)


def gdn_replay_accept_fold(d: Dims, buf_len, state_idx, accepted, status, stream=None):
    i32 = torch.int32
    _check_sizes(d, buf_len=buf_len, state_idx=state_idx, accepted=accepted, status=status)
    rc = load().gdn_replay_accept_fold(ctypes.byref(d), _ptr(buf_len, i32, "buf_len"),
                                       _ptr(state_idx, i32, "state_idx"),
                                       _ptr(accepted, i32, "accepted"), _ptr(status, i32, "status"),
                                       _stream(stream))
    _check("gdn_replay_accept_fold", rc)


def gdn_replay_accept(d: Dims, buf_len, state_idx, accepted, status, stream=None):
    i32 = torch.int32
    _check_sizes(d, buf_len=buf_len, state_idx=state_idx, accepted=accepted, status=status)
    rc = load().gdn_replay_accept(ctypes.byref(d), _ptr(buf_len, i32, "buf_len"),
                                  _ptr(state_idx, i32, "state_idx"),
                                  _ptr(accepted, i32, "accepted"), _ptr(status, i32, "status"),
                                  _stream(stream))
    _check("gdn_replay_accept", rc)


def gdn_replay_flush(d: Dims, state, state_idx, buf_k, buf_v, buf_g, buf_beta, buf_len, force,
                     status, stream=None):
    tin = _TORCH_IN.get(d.in_dtype)
    f32, i32 = torch.float32, torch.int32
    _check_sizes(d, state=state, state_idx=state_idx, buf_k=buf_k, buf_v=buf_v, buf_g=buf_g,
                 buf_beta=buf_beta, buf_len=buf_len, status=status)
    rc = load().gdn_replay_flush(
        ctypes.byref(d), _ptr(state, f32, "state"), _ptr(state_idx, i32, "state_idx"),
        _ptr(buf_k, tin, "buf_k"), _ptr(buf_v, tin, "buf_v"), _ptr(buf_g, f32, "buf_g"),
        _ptr(buf_beta, f32, "buf_beta"), _ptr(buf_len, i32, "buf_len"), int(bool(force)),
        _ptr(status, i32, "status"), _stream(stream))
    _check("gdn_replay_flush", rc)


def gdn_replay_advance_workspace(d: AdvanceDims) -> int:
    """Bytes of workspace that gdn_replay_advance needs for these dims."""
    n = load().gdn_replay_advance_workspace(ctypes.byref(d))
    _check("gdn_replay_advance_workspace", min(n, 0))
    return n


def gdn_replay_advance(d: AdvanceDims, state, state_idx, buf_len, chunk_len, fresh, q, k, v, g, beta, out, workspace,
                       status, stream=None):
    """Committed tokens over the checkpoint (include/gdnreplay.h).  q, k and v may be views of one projection's
    output; their strides are set in a copy of d."""
    tin = _TORCH_IN.get(d.in_dtype)
    if tin is None:
        raise GdnError("gdn_replay_advance", -3)
    d = AdvanceDims.from_buffer_copy(d)
    dev = state.get_device() if isinstance(state, torch.Tensor) else -1
    rows, tok = d.B * d.T, (d.B, d.T)
    pq, d.q_stride = _tokens(q, tok + (d.Hk, d.dk), tin, dev, "q")
    pk, d.k_stride = _tokens(k, tok + (d.Hk, d.dk), tin, dev, "k")
    pv, d.v_stride = _tokens(v, tok + (d.H, d.dv), tin, dev, "v")
    gate = tok + (d.H,)
    rc = load().gdn_replay_advance(
        ctypes.byref(d), _in(state, _F32, d.n_slot * d.H * d.dv * d.dk, "state"),
        None if state_idx is None else _in(state_idx, _I32, d.B, "state_idx", dev),
        None if buf_len is None else _in(buf_len, _I32, d.n_slot, "buf_len", dev),
        None if chunk_len is None else _in(chunk_len, _I32, d.B, "chunk_len", dev),
        None if fresh is None else _in(fresh, _I32, d.B, "fresh", dev), pq, pk, pv,
        _in(g, _F32, rows * d.H, "g", dev, gate), _in(beta, _F32, rows * d.H, "beta", dev, gate),
        _in(out, _F32, rows * d.H * d.dv, "out", dev, gate + (d.dv,)),
        None if workspace is None else _in(workspace, torch.uint8, 0, "workspace", dev),
        0 if workspace is None else workspace.numel(), _in(status, _I32, 1, "status", dev),
        _raw_stream(stream, dev))
    if rc:
        raise GdnError("gdn_replay_advance", rc)


class ReplayLayer:
    """Device-resident checkpoint, buffer and lengths of one GDN layer.

    ``init`` is a dict of CPU tensors with the layouts of ``include/gdnreplay.h``
    (state, state_idx, buf_k, buf_v, buf_g, buf_beta, buf_len); they are copied
    to ``device`` once.  A state_idx of None is the identity map (sequence b owns
    slot b).  The methods enqueue the library calls.
    """

    def __init__(self, dims: Dims, init: dict, device="cuda"):
        self.d = dims
        self.t = {n: None if init[n] is None else init[n].to(device).contiguous() for n in
                  ("state", "state_idx", "buf_k", "buf_v", "buf_g", "buf_beta", "buf_len")}
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._advances = {}

    def verify(self, q, k, v, g, beta, out, stream=None):
        t = self.t
        gdn_replay_verify(self.d, t["state"], t["state_idx"], t["buf_k"], t["buf_v"], t["buf_g"],
                          t["buf_beta"], t["buf_len"], q, k, v, g, beta, out, self.status, stream)

    def accept(self, accepted, stream=None):
        gdn_replay_accept(self.d, self.t["buf_len"], self.t["state_idx"], accepted, self.status,
                          stream)

    def flush(self, force=False, stream=None):
        t = self.t
        gdn_replay_flush(self.d, t["state"], t["state_idx"], t["buf_k"], t["buf_v"], t["buf_g"],
                         t["buf_beta"], t["buf_len"], force, self.status, stream)

    def verify_fold(self, q, k, v, g, beta, out, stream=None):
        t = self.t
        gdn_replay_verify_fold(self.d, t["state"], t["state_idx"], t["buf_k"], t["buf_v"],
                               t["buf_g"], t["buf_beta"], t["buf_len"], q, k, v, g, beta, out,
                               self.status, stream)

    def accept_fold(self, accepted, stream=None):
        gdn_replay_accept_fold(self.d, self.t["buf_len"], self.t["state_idx"], accepted,
                               self.status, stream)

    def _advance_dims(self, T, Hk):
        """The dims of an advance (strides of dense tensors) and its workspace's bytes; kept by the numbers they follow
        from, as a single token's call is mostly host work."""
        key = (T, Hk, bytes(self.d))
        got = self._advances.get(key)
        if got is None:
            d = self.d
            e = 16 // (2 if d.in_dtype == DTYPE_BF16 else 4)
            a = AdvanceDims(B=d.B, T=T, H=d.H, Hk=Hk, dk=d.dk, dv=d.dv, n_slot=d.n_slot, in_dtype=d.in_dtype, scale=d.scale,
                            flags=d.flags, q_stride=Hk * d.dk // e * e, k_stride=Hk * d.dk // e * e, v_stride=d.H * d.dv)
            if len(self._advances) >= 64:
                self._advances.clear()
            got = self._advances[key] = a, gdn_replay_advance_workspace(a)
        return got

    def advance_workspace(self, T, Hk=None):
        """A workspace for ``advance`` with up to T tokens per sequence and Hk key heads (None: as many as value
        heads), or None where none is needed.  Layers that run one after the other may share one."""
        _, n = self._advance_dims(T, self.d.H if Hk is None else Hk)
        return torch.empty(n, dtype=torch.uint8, device=self.status.device) if n else None

    def advance(self, q, k, v, g, beta, out, chunk_len=None, fresh=None, workspace=None, stream=None):
        """Committed tokens (a prompt, a chunk of one, a single token) over the checkpoint, in place: q, k
        [B, T, Hk, dk], v [B, T, H, dv] (views of one projection's output, say), g, beta [B, T, H], out fp32
        [B, T, H, dv]; chunk_len int32 [B] tokens in use (None: T); fresh int32 [B], not 0: the sequence
        starts from a zero state.  The sequences' buffers have to be empty (flush(force=True)).  Without
        ``workspace`` (advance_workspace) one is allocated for the call."""
        if q.dim() != 4 or k.dim() != 4:
            raise ValueError("q, k: expected [B, T, Hk, dk]")
        d, n = self._advance_dims(q.shape[1], k.shape[2])
        if n and workspace is None:
            with torch.cuda.stream(stream):
                workspace = torch.empty(n, dtype=torch.uint8, device=self.status.device)
        t = self.t
        gdn_replay_advance(d, t["state"], t["state_idx"], t["buf_len"], chunk_len, fresh, q, k, v, g, beta, out, workspace,
                           self.status, stream)


# ---------------------------------------------------------- non-replay baseline
def _check_nr_sizes(d: Dims, **tensors):
    B, H, dk, dv, T, n = d.B, d.H, d.dk, d.dv, d.T, d.n_slot
    need = {"state": n * H * dv * dk, "state_idx": B, "q": B * T * H * dk, "k": B * T * H * dk,
            "v": B * T * H * dv, "g": B * T * H, "beta": B * T * H, "out": B * T * H * dv,
            "snap": B * H * T * dv * dk, "accepted": B, "status": 1}
    for name, t in tensors.items():
        if isinstance(t, torch.Tensor) and t.numel() < need[name]:
            raise ValueError(f"{name}: needs at least {need[name]} elements for {d}, got {t.numel()}")


def gdn_nonreplay_verify(d: Dims, state, state_idx, q, k, v, g, beta, out, snap, status, stream=None):
    """The baseline without a buffer (include/gdnnonreplay.h): outputs of the draft
    block from the current state and the state after every draft token in ``snap``."""
    tin = _TORCH_IN.get(d.in_dtype)
    f32, i32 = torch.float32, torch.int32
    _check_nr_sizes(d, state=state, state_idx=state_idx, q=q, k=k, v=v, g=g, beta=beta, out=out,
                    snap=snap, status=status)
    rc = load().gdn_nonreplay_verify(
        ctypes.byref(d), _ptr(state, f32, "state"), _ptr(state_idx, i32, "state_idx"),
        _ptr(q, tin, "q"), _ptr(k, tin, "k"), _ptr(v, tin, "v"), _ptr(g, f32, "g"),
        _ptr(beta, f32, "beta"), _ptr(out, f32, "out"), _ptr(snap, f32, "snap"),
        _ptr(status, i32, "status"), _stream(stream))
    _check("gdn_nonreplay_verify", rc)


def gdn_nonreplay_accept(d: Dims, state, state_idx, snap, accepted, status, stream=None):
    """Restore by copy: the state after the accepted prefix (snapshot p - 1)."""
    f32, i32 = torch.float32, torch.int32
    _check_nr_sizes(d, state=state, state_idx=state_idx, snap=snap, accepted=accepted, status=status)
    rc = load().gdn_nonreplay_accept(
        ctypes.byref(d), _ptr(state, f32, "state"), _ptr(state_idx, i32, "state_idx"),
        _ptr(snap, f32, "snap"), _ptr(accepted, i32, "accepted"), _ptr(status, i32, "status"),
        _stream(stream))
    _check("gdn_nonreplay_accept", rc)


class NonReplayLayer:
    """Device-resident state of one GDN layer under the non-replay baseline, with
    the snapshot area its verify writes (B x H x T states).  ``snap`` may be shared
    between layers that are stepped one after the other."""

    def __init__(self, dims: Dims, state, state_idx, device="cuda", snap=None):
        self.d = dims
        self.state = state.to(device).contiguous()
        self.state_idx = None if state_idx is None else state_idx.to(device).contiguous()
        n = dims.B * dims.H * dims.T * dims.dv * dims.dk
        self.snap = torch.empty(n, dtype=torch.float32, device=device) if snap is None else snap
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def verify(self, q, k, v, g, beta, out, stream=None):
        gdn_nonreplay_verify(self.d, self.state, self.state_idx, q, k, v, g, beta, out, self.snap,
                             self.status, stream)

    def accept(self, accepted, stream=None):
        gdn_nonreplay_accept(self.d, self.state, self.state_idx, self.snap, accepted, self.status,
                             stream)


# ------------------------------------------------ causal convolution with rollback
def _conv_sizes(d: ConvDims) -> dict:
    return {"ring": d.n_slot * d.cap * d.D, "ring_pos": d.n_slot, "state_idx": d.B,
            "x": d.B * d.T * d.D, "weight": d.D * d.W, "bias": d.D, "y": d.B * d.T * d.D,
            "accepted": d.B, "status": 1}


def _check_conv_sizes(d: ConvDims, **tensors):
    need = _conv_sizes(d)
    for name, t in tensors.items():
        if isinstance(t, torch.Tensor) and t.numel() < need[name]:
            raise ValueError(f"{name}: needs at least {need[name]} elements for {d}, got {t.numel()}")


def gdn_conv_verify(d: ConvDims, ring, ring_pos, state_idx, x, weight, bias, y, status, stream=None):
    tin, tout = _TORCH_IN.get(d.in_dtype), _TORCH_IN.get(d.out_dtype)
    f32, i32 = torch.float32, torch.int32
    _check_conv_sizes(d, ring=ring, ring_pos=ring_pos, state_idx=state_idx, x=x, weight=weight,
                      bias=bias, y=y, status=status)
    rc = load().gdn_conv_verify(
        ctypes.byref(d), _ptr(ring, tin, "ring"), _ptr(ring_pos, i32, "ring_pos"),
        _ptr(state_idx, i32, "state_idx"), _ptr(x, tin, "x"), _ptr(weight, f32, "weight"),
        _ptr(bias, f32, "bias"), _ptr(y, tout, "y"), _ptr(status, i32, "status"), _stream(stream))
    _check("gdn_conv_verify", rc)


def gdn_conv_accept(d: ConvDims, ring_pos, state_idx, accepted, status, stream=None):
    i32 = torch.int32
    _check_conv_sizes(d, ring_pos=ring_pos, state_idx=state_idx, accepted=accepted, status=status)
    rc = load().gdn_conv_accept(ctypes.byref(d), _ptr(ring_pos, i32, "ring_pos"),
                                _ptr(state_idx, i32, "state_idx"), _ptr(accepted, i32, "accepted"),
                                _ptr(status, i32, "status"), _stream(stream))
    _check("gdn_conv_accept", rc)


def gdn_conv_advance(d: ConvDims, ring, ring_pos, state_idx, chunk_len, fresh, x, weight, bias, y, status, stream=None):
    """The convolution over committed tokens (include/gdnlayer.h); d.T tokens per sequence."""
    tin, tout = _TORCH_IN.get(d.in_dtype), _TORCH_IN.get(d.out_dtype)
    if tin is None or tout is None:
        raise GdnError("gdn_conv_advance", -3)
    dev = ring.get_device() if isinstance(ring, torch.Tensor) else -1
    n, block = d.B * d.T * d.D, (d.B, d.T, d.D)
    rc = load().gdn_conv_advance(
        ctypes.byref(d), _in(ring, tin, d.n_slot * d.cap * d.D, "ring"), _in(ring_pos, _I32, d.n_slot, "ring_pos", dev),
        None if state_idx is None else _in(state_idx, _I32, d.B, "state_idx", dev),
        None if chunk_len is None else _in(chunk_len, _I32, d.B, "chunk_len", dev),
        None if fresh is None else _in(fresh, _I32, d.B, "fresh", dev), _in(x, tin, n, "x", dev, block),
        _in(weight, _F32, d.D * d.W, "weight", dev), None if bias is None else _in(bias, _F32, d.D, "bias", dev),
        _in(y, tout, n, "y", dev, block), _in(status, _I32, 1, "status", dev), _raw_stream(stream, dev))
    if rc:
        raise GdnError("gdn_conv_advance", rc)


class ConvLayer:
    """Device-resident convolution ring, write positions, weight and bias of one
    layer (``init``: CPU tensors ring, pos, state_idx, weight, bias; a state_idx of
    None is the identity map)."""

    def __init__(self, dims: ConvDims, init: dict, device="cuda"):
        self.d = dims
        self.t = {n: None if init[n] is None else init[n].to(device).contiguous()
                  for n in ("ring", "pos", "state_idx", "weight")}
        self.t["bias"] = None if init.get("bias") is None else init["bias"].to(device).contiguous()
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def verify(self, x, y, stream=None):
        t = self.t
        gdn_conv_verify(self.d, t["ring"], t["pos"], t["state_idx"], x, t["weight"], t["bias"], y,
                        self.status, stream)

    def accept(self, accepted, stream=None):
        gdn_conv_accept(self.d, self.t["pos"], self.t["state_idx"], accepted, self.status, stream)

    def advance(self, x, y, chunk_len=None, fresh=None, stream=None):
        """Committed tokens (a prompt, a chunk of one, a single token): x, y [B, T, D], not overlapping; chunk_len int32 [B]
        tokens in use (None: T); fresh int32 [B], not 0: the sequence starts from a window of zeros."""
        if x.dim() != 3:
            raise ValueError(f"x: expected [B, T, D], got {tuple(x.shape)}")
        d, t = ConvDims.from_buffer_copy(self.d), self.t
        d.T = x.shape[1]
        gdn_conv_advance(d, t["ring"], t["pos"], t["state_idx"], chunk_len, fresh, x, t["weight"], t["bias"], y, self.status,
                         stream)


# ---------------------------------------------------- gated RMSNorm + E4M3 codes
def gdn_gated_rmsnorm_fp8(o, z, weight, eps: float, inv_scale: float, q, stream=None):
    """o fp32 [rows, d] (any shape whose last dim is d), z bf16/fp32 like o, weight fp32 [d],
    q uint8 like o (E4M3 codes)."""
    d = o.shape[-1]
    rows = o.numel() // d if d else 0
    if z.numel() != o.numel() or q.numel() != o.numel() or weight.numel() != d:
        raise ValueError("o, z and q must have the same number of elements; weight must have d")
    zt = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(z.dtype)
    if zt is None:
        raise TypeError(f"z: expected bfloat16 or float32, got {z.dtype}")
    rc = load().gdn_gated_rmsnorm_fp8(rows, d, _ptr(o, torch.float32, "o"), _ptr(z, None, "z"), zt,
                                      _ptr(weight, torch.float32, "weight"), float(eps),
                                      float(inv_scale), _ptr(q, torch.uint8, "q"), _stream(stream))
    _check("gdn_gated_rmsnorm_fp8", rc)


# ------------------------------------------ attention layers: paged cache and drafts
_I32, _F32 = torch.int32, torch.float32

# The current stream's handle without the Stream object that torch.cuda.current_stream()
# makes (3 us a call against 0.1); the object is the way where torch lacks the function.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _raw_stream(stream, index):
    """Handle of ``stream``, of the device's current one when None."""
    return _current_raw_stream(index) if stream is None else stream.cuda_stream


def _tokens(t, shape, dtype, index, name):
    """Address and token stride of a [B, T, heads, d] tensor that is dense within a token, its tokens
    evenly spaced."""
    B, T, heads, n = shape
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if t.get_device() != index or index < 0:
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor")
        raise ValueError(f"{name}: expected a tensor on the layer's device (cuda:{index}), got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    sb, st, sh, se = t.stride()
    if se != 1 or (heads > 1 and sh != n):
        raise ValueError(f"{name}: the heads of a token must be dense")
    if T == 1:
        st = sb if B > 1 else heads * n                  # a single token's stride says nothing
    elif B > 1 and sb != T * st:
        raise ValueError(f"{name}: tokens must be evenly spaced over the batch")
    return t.data_ptr(), st


def _in(t, dtype, n, name, index=None, shape=None):
    """Address of a dense tensor of dtype that holds at least n elements, on the CUDA device of that
    index (None: any) and in an order of extents that _fits ``shape``."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous():
        at = t.get_device()                             # (-1 for the CPU's)
        if at >= 0 and (index is None or at == index):
            # one comparison for the usual tensor; a host call of a short kernel is made of such checks
            if (shape is not None and t.shape == shape) or (t.numel() >= n and (shape is None or _fits(t.shape, shape))):
                return t.data_ptr()
    _ptr(t, dtype, name)                                # says what is wrong
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name}: expected a tensor on the cache's device (cuda:{index}), got {t.device}")
    if t.numel() < n:
        raise ValueError(f"{name}: needs at least {n} elements, got {t.numel()}")
    raise ValueError(f"{name}: expected shape {shape} or neighbouring extents of it in one, got {tuple(t.shape)}")


def _fits(got, shape):
    """Whether a dense tensor of extents ``got`` holds ``shape`` in row-major order: its extents behind the
    first are those of ``shape``, neighbours in one or not, extents of 1 anywhere; the first may be longer."""
    ends, n = {1}, 1                                    # elements behind each extent of shape
    for x in reversed(shape):
        n *= x
        ends.add(n)
    n = 1
    for x in reversed(got[1:]):
        n *= x
        if n not in ends:
            return False
    return True


class PagedCache:
    """Keys and values of the attention layers in pages, and the pages' bookkeeping
    (include/gdnattn.h).

    ``init`` is a dict of tensors k, v, block_table, seq_len, n_owned, ref, free_list and
    free_count with the header's layouts; they are moved to ``device`` once (a tensor that
    is there already is used as it is).  Without ``init`` every page is free and k and v are
    zeros.  The tensors are attributes; write into them, do not replace them.  ``status``
    collects GDN_STATUS_* bits: a row without free pages, say, is skipped on the device, and the
    calls after it refuse its tokens there (STATUS_BAD_PAGE).  Whoever fills the block table without
    ``reserve`` and ``fork`` sets n_owned as well: entries past it are not used.  The methods enqueue
    the library calls.
    """

    _FIELDS = ("k", "v", "block_table", "seq_len", "n_owned", "ref", "free_list", "free_count")

    def __init__(self, dims: PageDims, init: dict | None = None, device="cuda"):
        t, n = _TORCH_IN.get(dims.dtype), dims
        if t is None:
            raise TypeError(f"dtype: expected DTYPE_BF16 or DTYPE_F32, got {dims.dtype}")
        shape = {"k": (n.n_layer, n.n_page, n.Hkv, n.page, n.d), "block_table": (n.n_slot, n.max_pages),
                 "seq_len": (n.n_slot,), "n_owned": (n.n_slot,), "ref": (n.n_page,), "free_list": (n.n_page,),
                 "free_count": (1,)}
        shape["v"] = shape["k"]
        if init is None:
            init = {f: torch.zeros(shape[f], dtype=t if f in "kv" else torch.int32, device=device)
                    for f in self._FIELDS}
            init["block_table"].fill_(-1)
            init["free_list"].copy_(torch.arange(n.n_page - 1, -1, -1, dtype=torch.int32))
            init["free_count"].fill_(n.n_page)
        self._t = {}
        self.d = PageDims(**{f: getattr(dims, f) for f, _ in PageDims._fields_[:8]})
        for f in self._FIELDS:
            x = init[f].to(device).contiguous()
            if tuple(x.shape) != shape[f]:
                raise ValueError(f"{f}: expected shape {shape[f]}, got {tuple(x.shape)}")
            setattr(self.d, f, _ptr(x, t if f in "kv" else torch.int32, f) or None)
            self._t[f] = x
        self._c = ctypes.byref(self.d)
        dev = self._t["k"].device
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._status, self._index = self.status.data_ptr(), dev.index
        self._lib = load()

    def __getattr__(self, name):
        if name in PagedCache._FIELDS:
            return self._t[name]
        raise AttributeError(name)

    def _stream(self, stream):
        return _current_raw_stream(self._index) if stream is None else stream.cuda_stream

    def reserve(self, slots, extra: int, stream=None):
        """Room for ``extra`` tokens past seq_len in each of ``slots`` (int32)."""
        n = slots.numel()
        rc = self._lib.gdn_pages_reserve(self._c, n, _in(slots, _I32, n, "slots", self._index), extra,
                                         self._status, self._stream(stream))
        if rc:
            raise GdnError("gdn_pages_reserve", rc)

    def fork(self, src, dst, copies, stream=None):
        """Sequences ``dst`` become copies of ``src`` (int32 slots): full pages shared, the
        last page's rows copied in every layer.  ``copies`` int32 [n, 2] receives those pages."""
        n, s = src.numel(), self._stream(stream)
        c, at = _in(copies, _I32, 2 * n, "copies", self._index), self._index
        rc = self._lib.gdn_pages_fork(self._c, n, _in(src, _I32, n, "src", at), _in(dst, _I32, n, "dst", at), c,
                                      self._status, s)
        if rc:
            raise GdnError("gdn_pages_fork", rc)
        rc = self._lib.gdn_pages_copy(self._c, n, c, self._status, s)
        if rc:
            raise GdnError("gdn_pages_copy", rc)

    def release(self, slots, stream=None):
        """The pages of ``slots`` (int32) go back, as far as no other sequence holds them."""
        n = slots.numel()
        rc = self._lib.gdn_pages_release(self._c, n, _in(slots, _I32, n, "slots", self._index), self._status,
                                         self._stream(stream))
        if rc:
            raise GdnError("gdn_pages_release", rc)

    def accept(self, accepted, path=None, state_idx=None, new_len=None, stream=None, T=None):
        """Commit accepted[b] drafted tokens of each sequence: along ``path`` (int32 [B, T]),
        whose rows move to the front of the draft's in every layer, or, without one, the first
        accepted[b].  More than ``T`` (the draft's tokens per sequence; 64, the most there can be, when
        neither it nor a path says) are refused on the device (STATUS_BAD_ACCEPT).  The lengths go
        to ``new_len`` (seq_len when None)."""
        B, at = accepted.numel(), self._index
        if path is not None:
            if T is not None and T != path.shape[-1]:
                raise ValueError(f"path: expected {T} tokens per sequence, got {path.shape[-1]}")
            T = path.shape[-1]
        elif T is None:
            T = 64
        rc = self._lib.gdn_attn_accept(
            self._c, B, T, None if state_idx is None else _in(state_idx, _I32, B, "state_idx", at),
            None if path is None else _in(path, _I32, B * T, "path", at), _in(accepted, _I32, B, "accepted", at),
            self.d.seq_len if new_len is None else _in(new_len, _I32, self.d.n_slot, "new_len", at),
            self._status, self._stream(stream))
        if rc:
            raise GdnError("gdn_attn_accept", rc)


class AttnLayer:
    """One attention layer over a PagedCache: the staging of a draft block and its verify.

    ``rope``, ``q_weight``, ``k_weight`` (fp32 [d]) and ``cos_sin`` (fp32 [max_pos, rot]) serve
    ``stage`` alone.  state_idx (int32 [B]) maps rows to slots; None is the identity.  Unless a
    workspace is passed (layers that run one after the other may share one: ``other.workspace``), a verify's
    is allocated here, that of a chunk of more than 64 tokens with the first ``chunk`` or look at
    ``workspace``: a layer that only stages needs none.  ``status`` is the cache's.
    """

    def __init__(self, dims: AttnDims, cache: PagedCache, layer: int, rope: RopeDims | None = None,
                 q_weight=None, k_weight=None, cos_sin=None, state_idx=None, workspace=None):
        c = cache.d
        self._d, self.cache, self.layer, self.status = AttnDims.from_buffer_copy(dims), cache, layer, cache.status
        self._rope = None if rope is None else RopeDims.from_buffer_copy(rope)
        self._ref, self._B, self._rows = ctypes.byref(self._d), dims.B, dims.B * dims.T
        self._heads = self._rows * dims.Hq                      # rows of queries
        self._elems = self._heads * c.d
        self._tok, self._row = (dims.B, dims.T), (dims.B, dims.T, dims.Hq)
        self._vec, self._kv = self._row + (c.d,), self._tok + (c.Hkv, c.d)
        dev = cache.status.device
        need, later = 0, dims.T > 64
        if not later:
            need = cache._lib.gdn_attn_workspace(cache._c, self._ref)
            _check("gdn_attn_workspace", min(need, 0))
        self._chunk_need = None if later else need               # (a chunk of up to 64 tokens is a verify)
        self._index = at = cache._index
        self._to_allocate = workspace is None and later
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        self.state_idx = state_idx
        self._keep = (q_weight, k_weight, cos_sin, state_idx)    # the calls use their addresses
        self._take(workspace, need)
        self._idx = None if state_idx is None else _in(state_idx, _I32, dims.B, "state_idx", at)
        if rope is not None:
            self._w = (_in(q_weight, _F32, c.d, "q_weight", at), _in(k_weight, _F32, c.d, "k_weight", at),
                       None if cos_sin is None else _in(cos_sin, _F32, rope.max_pos * rope.rot, "cos_sin", at))
        self._dtype, self._stream, self._lib = _TORCH_IN[c.dtype], cache._stream, cache._lib

    @property
    def d(self):
        """A copy of the layer's dims."""
        return AttnDims.from_buffer_copy(self._d)

    def _take(self, workspace, need):
        self._ws, self._ws_bytes = _in(workspace, torch.uint8, need, "workspace", self._index) or None, workspace.numel()
        self._workspace = self._kept_workspace = workspace       # (the second holds on to it, whatever becomes of the first)

    def _chunk_workspace(self, stream=None):
        """Bytes that a chunk needs; allocates them, once, for a layer that was given no workspace."""
        need = self._chunk_need
        if need is None:
            need = self._lib.gdn_attn_chunk_workspace(self.cache._c, self._ref)
            _check("gdn_attn_chunk", min(need, 0))
            self._chunk_need = need
        if self._to_allocate:
            with torch.cuda.stream(stream):
                self._take(torch.empty(need, dtype=torch.uint8, device=self.status.device), need)
            self._to_allocate = False
        return need

    @property
    def workspace(self):
        """The layer's workspace; that of a chunk is allocated when it is first needed."""
        if self._to_allocate:
            try:
                self._chunk_workspace()
            except GdnError:                                     # (dims that stage takes and chunk does not: it has none)
                pass
        return self._workspace

    @workspace.setter
    def workspace(self, value):
        self._workspace = value

    def _block(self, t, shape, name):
        """Address and token stride of q, k or v: [B, T, heads, d], dense within a token, the
        tokens evenly spaced."""
        B, T, heads, n = shape
        if t.shape != shape:
            raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
        if t.get_device() != self._index:
            if not t.is_cuda:
                raise ValueError(f"{name}: expected a CUDA tensor")
            raise ValueError(f"{name}: expected a tensor on the cache's device (cuda:{self._index}), got {t.device}")
        if t.dtype is not self._dtype:
            raise TypeError(f"{name}: expected {self._dtype}, got {t.dtype}")
        sb, st, sh, se = t.stride()
        if se != 1 or (heads > 1 and sh != n):
            raise ValueError(f"{name}: the heads of a token must be dense")
        if T == 1:
            st = sb if B > 1 else heads * n              # a single token's stride says nothing
        elif B > 1 and sb != T * st:
            raise ValueError(f"{name}: tokens must be evenly spaced over the batch")
        return t.data_ptr(), st

    def stage(self, q, k, v, q_out, pos=None, draft_len=None, stream=None):
        """Norm and rotate q [B, T, Hq, d] into ``q_out`` and k [B, T, Hkv, d] into the cache's
        draft rows, v beside it.  q, k and v may be views of one projection's output."""
        if self._rope is None:
            raise ValueError("stage: this layer was made without rope and norm weights")
        r = RopeDims.from_buffer_copy(self._rope)
        pq, r.q_stride = self._block(q, self._vec, "q")
        pk, r.k_stride = self._block(k, self._kv, "k")
        pv, r.v_stride = self._block(v, self._kv, "v")
        wq, wk, tab = self._w
        cache, at = self.cache, self._index
        rc = self._lib.gdn_attn_stage(
            cache._c, self.layer, self._ref, ctypes.byref(r), self._idx,
            None if draft_len is None else _in(draft_len, _I32, self._B, "draft_len", at), pq, pk, pv,
            None if pos is None else _in(pos, _I32, self._rows, "pos", at, self._tok), wq, wk, tab,
            _in(q_out, self._dtype, self._elems, "q_out", at, self._vec), cache._status, self._stream(stream))
        if rc:
            raise GdnError("gdn_attn_stage", rc)

    def build_tree(self, parent, tree, pos=None, draft_len=None, stream=None):
        """Ancestor words ``tree`` (int64 [B, T]) and rotation positions ``pos`` (int32 [B, T])
        of a token tree given by its parents (int32 [B, T])."""
        n, tok, at = self._rows, self._tok, self._index
        rc = self._lib.gdn_tree_build(
            self.cache._c, self._ref, self._idx,
            None if draft_len is None else _in(draft_len, _I32, self._B, "draft_len", at),
            _in(parent, _I32, n, "parent", at, tok), _in(tree, torch.int64, n, "tree", at, tok),
            None if pos is None else _in(pos, _I32, n, "pos", at, tok), self.cache._status, self._stream(stream))
        if rc:
            raise GdnError("gdn_tree_build", rc)

    def verify(self, q, out, lse=None, tree=None, draft_len=None, stream=None):
        """Attention of the block's rows q [B, T, Hq, d] over the cache into ``out`` (and
        ``lse`` fp32 [B, T, Hq]); ``tree`` int64 [B, T] ancestor words, None: a chain.  Neighbouring
        extents may be one ([B, T, Hq d]), and the first may be longer."""
        t, e, cache, at = self._dtype, self._elems, self.cache, self._index
        rc = self._lib.gdn_attn_verify(
            cache._c, self.layer, self._ref, self._idx,
            None if draft_len is None else _in(draft_len, _I32, self._B, "draft_len", at),
            _in(q, t, e, "q", at, self._vec),
            None if tree is None else _in(tree, torch.int64, self._rows, "tree", at, self._tok),
            _in(out, t, e, "out", at, self._vec),
            None if lse is None else _in(lse, _F32, self._heads, "lse", at, self._row), self._ws, self._ws_bytes,
            cache._status, self._stream(stream))
        if rc:
            raise GdnError("gdn_attn_verify", rc)

    def chunk(self, q, out, lse=None, chunk_len=None, stream=None):
        """Causal attention of a chunk of new tokens (a prompt, a part of one), staged already: q [B, T, Hq, d]
        over the committed tokens and the chunk's own into ``out`` (and ``lse`` fp32 [B, T, Hq]).  chunk_len
        int32 [B]: tokens in use (None: T, any number that the layer was made for).  seq_len does not move:
        accept the chunk, or write the new lengths, afterwards.  bf16 chunks of more than 64 tokens round each softmax weight to bf16
        before the product with the values, unless the layer's dims have FLAG_TWO_TERMS; up to 64 are a verify, which keeps two terms."""
        if self._chunk_need is None or self._to_allocate or self._ws_bytes < self._chunk_need:
            need = self._chunk_workspace(stream)
            if self._ws_bytes < need:
                raise ValueError(f"chunk: needs a workspace of at least {need} bytes, got {self._ws_bytes}")
        t, e, cache, at = self._dtype, self._elems, self.cache, self._index
        rc = self._lib.gdn_attn_chunk(
            cache._c, self.layer, self._ref, self._idx,
            None if chunk_len is None else _in(chunk_len, _I32, self._B, "chunk_len", at),
            _in(q, t, e, "q", at, self._vec), _in(out, t, e, "out", at, self._vec),
            None if lse is None else _in(lse, _F32, self._heads, "lse", at, self._row), self._ws, self._ws_bytes,
            cache._status, self._stream(stream))
        if rc:
            raise GdnError("gdn_attn_chunk", rc)


# ------------------------------------------------------ drafted tokens against the target
class DraftSampler:
    """Speculative sampling: which drafted tokens of a block the target accepts, and the next token
    (include/gdndraft.h).  ``status`` int32 [1] collects GDN_STATUS_* bits."""

    def __init__(self, dims: DraftDims, device="cuda"):
        self.d = DraftDims.from_buffer_copy(dims)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._lib, self._index = load(), self.status.get_device()

    def _table(self, t, name):
        """Address and row stride of probabilities [B, T, V], dense within a row, rows evenly spaced."""
        d = self.d
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor")
        if t.shape != (d.B, d.T, d.V):
            raise ValueError(f"{name}: expected shape {(d.B, d.T, d.V)}, got {tuple(t.shape)}")
        if t.get_device() != self._index:
            raise ValueError(f"{name}: expected a tensor on cuda:{self._index}, got {t.device}")
        if t.dtype is not _F32:
            raise TypeError(f"{name}: expected torch.float32, got {t.dtype}")
        sb, st, sv = t.stride()
        if d.T == 1:
            st = sb if d.B > 1 else d.V
        if (d.V > 1 and sv != 1) or (d.B > 1 and d.T > 1 and sb != d.T * st):
            raise ValueError(f"{name}: rows must be dense and evenly spaced over the batch")
        return t.data_ptr(), st

    def accept(self, tokens, probs, u, accepted, next_token, draft=None, parent=None, path=None, draft_len=None,
               stream=None):
        """tokens int32 [B, T], of which token 0 is decided already; probs fp32 [B, T, V] the target's
        distribution after each token, draft fp32 [B, T, V] the drafter's that its children were drawn from (None: a
        drafter certain of its tokens); u fp32 [B, T] uniform in [0, 1).  parent int32 [B, T] as for build_tree
        (None: a chain).  Writes accepted int32 [B] (token 0 counted), next_token int32 [B] and path int32 [B, T]
        (the accepted tokens' numbers, then -1; a chain needs none): what the layers' accepts take."""
        d, at, n = DraftDims.from_buffer_copy(self.d), self._index, self.d.B * self.d.T
        tok = (d.B, d.T)
        pp, d.p_stride = self._table(probs, "probs")
        pq, d.q_stride = (None, 0) if draft is None else self._table(draft, "draft")
        rc = self._lib.gdn_draft_accept(
            ctypes.byref(d), _in(tokens, _I32, n, "tokens", at, tok),
            None if parent is None else _in(parent, _I32, n, "parent", at, tok), pp, pq, _in(u, _F32, n, "u", at, tok),
            None if draft_len is None else _in(draft_len, _I32, d.B, "draft_len", at),
            _in(accepted, _I32, d.B, "accepted", at), _in(next_token, _I32, d.B, "next_token", at),
            None if path is None else _in(path, _I32, n, "path", at, tok), self.status.data_ptr(), _raw_stream(stream, at))
        if rc:
            raise GdnError("gdn_draft_accept", rc)
