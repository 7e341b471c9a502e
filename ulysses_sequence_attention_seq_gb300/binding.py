"""ctypes binding of libulysses.so (include/ulysses.h): argument marshalling only.

Every function here has the name of the C entry point it calls and takes
torch tensors in place of raw pointers.  Nothing here computes: every step of
the path runs in the library's CUDA kernels.  If the library is missing the
first call raises; there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# ULYSSES_LIB selects another build of the library (the range-checked one).
LIB_PATH = os.environ.get("ULYSSES_LIB") or os.path.join(_HERE, "_build", "libulysses.so")
_lib = None

BF16, FP32 = 0, 1
OK = 0
STATUS_FWD_TIMEOUT, STATUS_BWD_TIMEOUT, STATUS_ROPE_TABLE, STATUS_SMEM_ALIGN, STATUS_BOUNDS = 1, 2, 4, 8, 16
STATUS_MASK = 32

EXPORTS = ("ulysses_validate", "ulysses_workspace_bytes", "ulysses_workspace_init",
           "ulysses_read_status", "ulysses_pack_qkv", "ulysses_attn_fwd", "ulysses_unpack_out",
           "ulysses_attn_bwd", "ulysses_attn_fwd_folded", "ulysses_attn_bwd_folded", "ulysses_status_string",
           "ulysses_qk_norm_pack", "ulysses_qk_norm_bwd", "ulysses_mask_bytes", "ulysses_mask_build",
           "ulysses_attn_fwd_mod", "ulysses_attn_bwd_mod")


class UlyssesError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed with {code}: {lib().ulysses_status_string(code).decode()}")


class CProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("S", ctypes.c_int), ("hidden", ctypes.c_int),
                ("n_head", ctypes.c_int), ("n_kv_head", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("P", ctypes.c_int), ("causal", ctypes.c_int), ("dtype", ctypes.c_int),
                ("use_rope", ctypes.c_int), ("rope_base", ctypes.c_float),
                ("softmax_scale", ctypes.c_float), ("ring", ctypes.c_int)]


@dataclasses.dataclass(frozen=True)
class Problem:
    """Mirror of ``ulysses_problem``."""
    B: int
    S: int
    hidden: int
    n_head: int
    n_kv_head: int
    head_dim: int
    P: int
    causal: bool = True
    dtype: int = BF16
    use_rope: bool = True
    rope_base: float = 10000.0
    softmax_scale: float = 0.0
    ring: int = 1  # ring positions of the Ulysses x ring hybrid (1: plain Ulysses)

    @classmethod
    def from_workload(cls, w) -> "Problem":
        return cls(B=w.B, S=w.S, hidden=w.hidden, n_head=w.n_head, n_kv_head=w.n_kv_head,
                   head_dim=w.head_dim, P=w.P, causal=w.causal,
                   dtype=BF16 if w.dtype == "bf16" else FP32, use_rope=w.use_rope,
                   rope_base=w.rope_base, ring=getattr(w, "ring", 1))

    def c(self) -> CProblem:
        return CProblem(self.B, self.S, self.hidden, self.n_head, self.n_kv_head, self.head_dim,
                        self.P, int(self.causal), self.dtype, int(self.use_rope),
                        float(self.rope_base), float(self.softmax_scale), int(self.ring))

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == BF16 else torch.float32

    @property
    def Sl(self):
        return self.S // self.P

    @property
    def Pu(self):
        """Ranks of one ring position (the All-to-All group): P / ring."""
        return self.P // max(self.ring, 1)

    @property
    def Cs(self):
        """Tokens a head-layout buffer holds: S / ring (S for plain Ulysses)."""
        return self.S // max(self.ring, 1)

    @property
    def hp(self):
        return self.n_head // self.Pu

    @property
    def kvp(self):
        """kv-heads a rank holds in head layout: n_kv_head / Pu, or one when
        n_kv_head < Pu (each kv-head then replicated to Pu / n_kv_head ranks)."""
        return self.n_kv_head // self.Pu if self.n_kv_head >= self.Pu else 1

    def __getstate__(self):
        """The fields alone: what calls have worked out (_facts) holds addresses of
        this process and stays out of copies and pickles."""
        return {k: v for k, v in self.__dict__.items() if k != "_facts"}

    def scale(self) -> float:
        return self.softmax_scale if self.softmax_scale > 0 else 1.0 / math.sqrt(self.head_dim)


class CScoreMod(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("mask_bytes", ctypes.c_size_t)]


@dataclasses.dataclass(frozen=True)
class ScoreMod:
    """Mirror of ``ulysses_score_mod``: scores capped at ``softcap`` by tanh (0:
    not), ``-slopes[h] * |i - k|`` added ([n_head] float32, on a 16-byte boundary:
    clone a slice), keys by the plan in ``mask`` (a byte tensor built by
    ulysses_mask_build)."""
    softcap: float = 0.0
    slopes: Optional[torch.Tensor] = None
    mask: Optional[torch.Tensor] = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() first "
                               "(the library has no non-CUDA fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp, P, sz = ctypes.c_void_p, ctypes.POINTER(CProblem), ctypes.c_size_t
        L.ulysses_validate.argtypes = [P]
        L.ulysses_workspace_bytes.argtypes = [P, ctypes.c_int]
        L.ulysses_workspace_bytes.restype = sz
        L.ulysses_workspace_init.argtypes = [P, vp, sz, vp]
        L.ulysses_read_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
        L.ulysses_read_status_async.argtypes = [vp, vp, vp]
        L.ulysses_pack_qkv.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_unpack_out.argtypes = [P, vp, vp, vp]
        L.ulysses_attn_fwd_folded.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd_folded.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.ulysses_noalloc_read_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
        L.ulysses_attn_bwd_prepare.argtypes = [P, vp, vp, vp, vp, sz, vp]
        L.ulysses_qkv_proj_pack.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_out_proj_unpack.argtypes = [P, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_selftest_wait_timeout.argtypes = [vp, sz, ctypes.c_ulonglong, vp]
        L.ulysses_selftest_ex2_rate.argtypes = [vp, sz, ctypes.POINTER(ctypes.c_longlong),
                                                ctypes.POINTER(ctypes.c_int), vp]
        L.ulysses_attn_bwd_dkdv.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd_dq.argtypes = [P, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd_fused.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd_dkdvq.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd_dq_finish.argtypes = [P, vp, vp, sz, vp]
        L.ulysses_attn_bwd_ds.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd_dkdv_ds.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd_dq_ds.argtypes = [P, vp, vp, vp, sz, vp]
        f32, M = ctypes.c_float, ctypes.POINTER(CScoreMod)
        L.ulysses_qk_norm_pack.argtypes = [P, vp, vp, vp, vp, vp, f32, vp, sz, vp, vp, vp, vp, sz, vp]
        L.ulysses_qk_norm_bwd.argtypes = [P, vp, vp, vp, vp, f32, vp, sz, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ulysses_mask_bytes.argtypes = [P]
        L.ulysses_mask_bytes.restype = sz
        L.ulysses_mask_build.argtypes = [P, vp, vp, ctypes.c_int, vp, sz, vp]
        L.ulysses_attn_fwd_mod.argtypes = [P, vp, vp, vp, M, vp, vp, vp, sz, vp]
        L.ulysses_attn_bwd_mod.argtypes = [P, vp, vp, vp, vp, vp, vp, M, vp, vp, vp, vp, sz, vp]
        L.ulysses_status_string.argtypes = [ctypes.c_int]
        L.ulysses_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libulysses must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, rc: int):
    if rc != OK:
        raise UlyssesError(fn, rc)


def ulysses_validate(prob: Problem) -> int:
    return lib().ulysses_validate(ctypes.byref(prob.c()))


def ulysses_workspace_bytes(prob: Problem, phase: int) -> int:
    return lib().ulysses_workspace_bytes(ctypes.byref(prob.c()), phase)


def ulysses_workspace_init(prob: Problem, ws: torch.Tensor, stream=None):
    _check("ulysses_workspace_init",
           lib().ulysses_workspace_init(ctypes.byref(prob.c()), _ptr(ws), ws.numel() * ws.element_size(),
                                        _stream(stream)))


def ulysses_read_status(ws: torch.Tensor, stream=None) -> int:
    out = ctypes.c_uint32(0)
    _check("ulysses_read_status", lib().ulysses_read_status(_ptr(ws), ctypes.byref(out), _stream(stream)))
    return out.value


def ulysses_read_status_async(ws: torch.Tensor, out: torch.Tensor, stream=None):
    """Enqueue a copy of the status word into `out` (a pinned uint32/int32
    host tensor of at least one element) on the stream; no synchronisation."""
    if out.device.type != "cpu" or out.element_size() != 4 or out.numel() < 1:
        raise ValueError("out must be a 4-byte host tensor")
    _check("ulysses_read_status_async", lib().ulysses_read_status_async(_ptr(ws), _ptr(out), _stream(stream)))


def ulysses_pack_qkv(prob, q_seq, k_seq, v_seq, q_head, k_head, v_head, ws, stream=None):
    _check("ulysses_pack_qkv", lib().ulysses_pack_qkv(
        ctypes.byref(prob.c()), _ptr(q_seq), _ptr(k_seq), _ptr(v_seq), _ptr(q_head), _ptr(k_head),
        _ptr(v_head), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_attn_fwd(prob, q_head, k_head, v_head, o_head, lse, ws, stream=None):
    _check("ulysses_attn_fwd", lib().ulysses_attn_fwd(
        ctypes.byref(prob.c()), _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(o_head), _ptr(lse),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_attn_fwd_folded(prob, q_seq, k_seq, v_seq, o_seq, lse, ws, stream=None):
    _check("ulysses_attn_fwd_folded", lib().ulysses_attn_fwd_folded(
        ctypes.byref(prob.c()), _ptr(q_seq), _ptr(k_seq), _ptr(v_seq), _ptr(o_seq), _ptr(lse),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_attn_bwd_folded(prob, q_seq, k_seq, v_seq, o_seq, lse, do_seq, dq_seq, dk_seq, dv_seq, ws,
                            stream=None):
    """The folded backward: q, k, v, O and dO read in sequence layout, the
    gradients written in sequence layout (RoPE off, S/P % 128 == 0)."""
    _check("ulysses_attn_bwd_folded", lib().ulysses_attn_bwd_folded(
        ctypes.byref(prob.c()), _ptr(q_seq), _ptr(k_seq), _ptr(v_seq), _ptr(o_seq), _ptr(lse), _ptr(do_seq),
        _ptr(dq_seq), _ptr(dk_seq), _ptr(dv_seq), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_unpack_out(prob, o_head, o_seq, stream=None):
    _check("ulysses_unpack_out", lib().ulysses_unpack_out(
        ctypes.byref(prob.c()), _ptr(o_head), _ptr(o_seq), _stream(stream)))


def ulysses_attn_bwd(prob, q_head, k_head, v_head, o_head, lse, do_seq, dq_seq, dk_seq, dv_seq, ws,
                     stream=None):
    _check("ulysses_attn_bwd", lib().ulysses_attn_bwd(
        ctypes.byref(prob.c()), _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(o_head), _ptr(lse),
        _ptr(do_seq), _ptr(dq_seq), _ptr(dk_seq), _ptr(dv_seq), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def ulysses_attn_bwd_prepare(prob, o_head, lse, do_seq, ws, stream=None):
    """Step 1 of the backward: dO seq -> head, delta and the rescaled LSE into ws."""
    _check("ulysses_attn_bwd_prepare", lib().ulysses_attn_bwd_prepare(
        ctypes.byref(prob.c()), _ptr(o_head), _ptr(lse), _ptr(do_seq), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_attn_bwd_dkdv(prob, q_head, k_head, v_head, dk_seq, dv_seq, ws, stream=None):
    """Step 2 of the backward: dK, dV and their head -> seq All-to-All."""
    _check("ulysses_attn_bwd_dkdv", lib().ulysses_attn_bwd_dkdv(
        ctypes.byref(prob.c()), _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(dk_seq), _ptr(dv_seq),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_attn_bwd_dq(prob, q_head, k_head, v_head, dq_seq, ws, stream=None):
    """Step 3 of the backward: dQ and its head -> seq All-to-All."""
    _check("ulysses_attn_bwd_dq", lib().ulysses_attn_bwd_dq(
        ctypes.byref(prob.c()), _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(dq_seq), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_attn_bwd_fused(prob, q_head, k_head, v_head, o_head, lse, do_seq, dq_seq, dk_seq, dv_seq, ws,
                           stream=None):
    """The backward with dQ accumulated in the dK/dV loop (phase-2 workspace)."""
    _check("ulysses_attn_bwd_fused", lib().ulysses_attn_bwd_fused(
        ctypes.byref(prob.c()), _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(o_head), _ptr(lse),
        _ptr(do_seq), _ptr(dq_seq), _ptr(dk_seq), _ptr(dv_seq), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def ulysses_attn_bwd_dkdvq(prob, q_head, k_head, v_head, dk_seq, dv_seq, ws, stream=None):
    """Fused step 2: dK, dV and the dQ shares added into the workspace accumulator."""
    _check("ulysses_attn_bwd_dkdvq", lib().ulysses_attn_bwd_dkdvq(
        ctypes.byref(prob.c()), _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(dk_seq), _ptr(dv_seq),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_attn_bwd_dq_finish(prob, dq_seq, ws, stream=None):
    """Fused step 3: dQ from the accumulator into sequence layout (accumulator re-zeroed)."""
    _check("ulysses_attn_bwd_dq_finish", lib().ulysses_attn_bwd_dq_finish(
        ctypes.byref(prob.c()), _ptr(dq_seq), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_attn_bwd_ds(prob, q_head, k_head, v_head, o_head, lse, do_seq, dq_seq, dk_seq, dv_seq, ws,
                        stream=None):
    """The backward with every tile pair's dS stored and dQ read back from it
    (phase-3 workspace)."""
    _check("ulysses_attn_bwd_ds", lib().ulysses_attn_bwd_ds(
        ctypes.byref(prob.c()), _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(o_head), _ptr(lse),
        _ptr(do_seq), _ptr(dq_seq), _ptr(dk_seq), _ptr(dv_seq), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def ulysses_attn_bwd_dkdv_ds(prob, q_head, k_head, v_head, dk_seq, dv_seq, ws, stream=None):
    """dS-store step 2: dK, dV, and every tile pair's dS into the workspace."""
    _check("ulysses_attn_bwd_dkdv_ds", lib().ulysses_attn_bwd_dkdv_ds(
        ctypes.byref(prob.c()), _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(dk_seq), _ptr(dv_seq),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_attn_bwd_dq_ds(prob, k_head, dq_seq, ws, stream=None):
    """dS-store step 3: dQ from the stored dS tiles and K, in sequence layout."""
    _check("ulysses_attn_bwd_dq_ds", lib().ulysses_attn_bwd_dq_ds(
        ctypes.byref(prob.c()), _ptr(k_head), _ptr(dq_seq), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def ulysses_qkv_proj_pack(prob, x_seq, w_qkv, b_qkv, q_head, k_head, v_head, ws, stream=None):
    """QKV projection of the sequence-sharded activations with the pack and
    RoPE fused (b_qkv may be None)."""
    _check("ulysses_qkv_proj_pack", lib().ulysses_qkv_proj_pack(
        ctypes.byref(prob.c()), _ptr(x_seq), _ptr(w_qkv), None if b_qkv is None else _ptr(b_qkv),
        _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_out_proj_unpack(prob, o_head, w_o, b_o, y_seq, ws, stream=None):
    """Output projection of the head-layout attention output with the unpack
    folded into its loads (b_o may be None)."""
    _check("ulysses_out_proj_unpack", lib().ulysses_out_proj_unpack(
        ctypes.byref(prob.c()), _ptr(o_head), _ptr(w_o), None if b_o is None else _ptr(b_o), _ptr(y_seq),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ulysses_selftest_wait_timeout(ws, limit_ns, stream=None):
    """A bounded wait that is made to run out: sets the forward-timeout bit of
    the workspace status word after limit_ns, without any fault."""
    _check("ulysses_selftest_wait_timeout", lib().ulysses_selftest_wait_timeout(
        _ptr(ws), ws.numel() * ws.element_size(), int(limit_ns), _stream(stream)))


def ulysses_selftest_ex2_rate(stream=None) -> float:
    """Measured base-2 exponentials per SM per cycle (synchronizes)."""
    cyc = torch.zeros(1, dtype=torch.int64, device="cuda")
    n, sms = ctypes.c_longlong(0), ctypes.c_int(0)
    _check("ulysses_selftest_ex2_rate", lib().ulysses_selftest_ex2_rate(
        _ptr(cyc), 8, ctypes.byref(n), ctypes.byref(sms), _stream(stream)))
    torch.cuda.synchronize()
    return n.value / (sms.value * float(cyc.item()))


def ulysses_attn_bwd_noalloc(prob, q_head, k_head, v_head, o_head, lse, do_seq, dq_seq, dk_seq,
                             dv_seq, stream=None):
    """The backward without a workspace (for callers that cannot allocate):
    scratch comes from the library's fixed 32 MiB device array."""
    _check("ulysses_attn_bwd_noalloc", lib().ulysses_attn_bwd_noalloc(
        ctypes.byref(prob.c()), _ptr(q_head), _ptr(k_head), _ptr(v_head), _ptr(o_head), _ptr(lse),
        _ptr(do_seq), _ptr(dq_seq), _ptr(dk_seq), _ptr(dv_seq), _stream(stream)))


def ulysses_noalloc_read_status(stream=None) -> int:
    """Status word of the noalloc backward's scratch array (waits for the stream)."""
    out = ctypes.c_uint32(0)
    _check("ulysses_noalloc_read_status", lib().ulysses_noalloc_read_status(ctypes.byref(out), _stream(stream)))
    return out.value


# ------------------------------------------- query/key norms, modified scores
#
# The C entry points cannot see sizes, types or devices: these functions check
# them (a tensor that is too small would be read past its end) and launch on
# the tensors' device.  Short calls are bound by this host code, so it is kept
# to one pass over the arguments; what depends on the problem alone is worked
# out once per Problem.

class _Facts:
    """The C struct of a problem and the element counts of its tensors."""
    __slots__ = ("ref", "dtype", "q_seq", "k_seq", "q_head", "k_head", "lse", "w", "slopes", "rows", "_c")

    def __init__(self, p: Problem):
        self._c = p.c()
        self.ref = ctypes.byref(self._c)
        code = lib().ulysses_validate(self.ref)
        if code != OK:
            raise UlyssesError("ulysses_validate", code)
        self.dtype = p.torch_dtype
        tok = p.B * p.S
        self.q_seq = self.q_head = tok * p.n_head * p.head_dim
        self.k_seq = tok * p.n_kv_head * p.head_dim
        self.k_head = p.P * p.B * p.Cs * p.kvp * p.head_dim
        self.lse, self.w, self.slopes, self.rows = tok * p.n_head, p.head_dim, p.n_head, tok


def _facts(prob: Problem) -> _Facts:
    f = prob.__dict__.get("_facts")
    if f is None:
        f = _Facts(prob)
        object.__setattr__(prob, "_facts", f)
    return f


def _wrong(name, t, dtype, numel, dev):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, other tensors of the call on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have {numel} elements, not {tuple(t.shape)}")


def _at(name, t, dtype, numel, dev):
    """The address of a checked tensor."""
    if t.dtype is not dtype or t.numel() != numel or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        _wrong(name, t, dtype, numel, dev)
    return t.data_ptr()


def _opt(name, t, dtype, numel, dev):
    return None if t is None else _at(name, t, dtype, numel, dev)


def _bytes(name, t, dev):
    """The address and size of a byte tensor (a workspace or a mask plan)."""
    if t is None:
        return None, 0
    n = t.numel()
    return _at(name, t, torch.uint8, n, dev), n


def _launch(fn, dev, stream, *args):
    """The entry point on the given stream, or `dev`'s current one, with `dev` current."""
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    call = getattr(lib(), fn)
    if torch.cuda.current_device() == dev:
        rc = call(*args, stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = call(*args, stream.cuda_stream)
    if rc != OK:
        raise UlyssesError(fn, rc)


def _device(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("the call's tensors must be CUDA tensors: the first one is not a CUDA tensor")
    return dev


def ulysses_qk_norm_pack(prob, q_seq, k_seq, v_seq, q_weight, k_weight, eps, mask, q_head, k_head, v_head, ws,
                         stream=None):
    """Pack with the RMS norm of every q and k head before the rotation
    (weights [head_dim] or None; mask: a mask plan or None)."""
    f = _facts(prob)
    dt, d = f.dtype, _device(q_seq)
    m, nm = _bytes("mask", mask, d)
    w, nw = _bytes("ws", ws, d)
    _launch("ulysses_qk_norm_pack", d, stream, f.ref, _at("q_seq", q_seq, dt, f.q_seq, d),
            _at("k_seq", k_seq, dt, f.k_seq, d), _at("v_seq", v_seq, dt, f.k_seq, d),
            _opt("q_weight", q_weight, dt, f.w, d), _opt("k_weight", k_weight, dt, f.w, d), eps, m, nm,
            _at("q_head", q_head, dt, f.q_head, d), _at("k_head", k_head, dt, f.k_head, d),
            _at("v_head", v_head, dt, f.k_head, d), w, nw)


def ulysses_qk_norm_bwd(prob, q_seq, k_seq, q_weight, k_weight, eps, dqn_seq, dkn_seq, dq_seq, dk_seq, dq_weight,
                        dk_weight, ws, mask=None, stream=None):
    """Backward of the norm: dqn_seq, dkn_seq (the attention backward's dq_seq,
    dk_seq) to the gradients of its inputs and, unless None, of its weights
    ([head_dim] float32)."""
    f = _facts(prob)
    dt, d = f.dtype, _device(q_seq)
    m, nm = _bytes("mask", mask, d)
    w, nw = _bytes("ws", ws, d)
    _launch("ulysses_qk_norm_bwd", d, stream, f.ref, _at("q_seq", q_seq, dt, f.q_seq, d),
            _at("k_seq", k_seq, dt, f.k_seq, d), _opt("q_weight", q_weight, dt, f.w, d),
            _opt("k_weight", k_weight, dt, f.w, d), eps, m, nm, _at("dqn_seq", dqn_seq, dt, f.q_seq, d),
            _at("dkn_seq", dkn_seq, dt, f.k_seq, d), _at("dq_seq", dq_seq, dt, f.q_seq, d),
            _at("dk_seq", dk_seq, dt, f.k_seq, d), _opt("dq_weight", dq_weight, torch.float32, f.w, d),
            _opt("dk_weight", dk_weight, torch.float32, f.w, d), w, nw)


def ulysses_mask_bytes(prob: Problem) -> int:
    return lib().ulysses_mask_bytes(ctypes.byref(prob.c()))


def ulysses_mask_build(prob, doc, prefix, window, mask, stream=None):
    """Build the mask plan `mask` (a uint8 tensor of ulysses_mask_bytes) from
    document ids and prefix lengths ([B, S] int32 or None) and a window (0: none)."""
    f = _facts(prob)
    d = _device(mask)
    m, nm = _bytes("mask", mask, d)
    _launch("ulysses_mask_build", d, stream, f.ref, _opt("doc", doc, torch.int32, f.rows, d),
            _opt("prefix", prefix, torch.int32, f.rows, d), int(window), m, nm)


def _mod(f: _Facts, mod: ScoreMod, d: int) -> CScoreMod:
    m, nm = _bytes("mask", mod.mask, d)
    return CScoreMod(mod.softcap, _opt("slopes", mod.slopes, torch.float32, f.slopes, d), m, nm)


def ulysses_attn_fwd_mod(prob, q_head, k_head, v_head, mod: ScoreMod, o_head, lse, ws, stream=None):
    """Attention with capped, biased and masked scores (ScoreMod)."""
    f = _facts(prob)
    dt, d = f.dtype, _device(q_head)
    w, nw = _bytes("ws", ws, d)
    _launch("ulysses_attn_fwd_mod", d, stream, f.ref, _at("q_head", q_head, dt, f.q_head, d),
            _at("k_head", k_head, dt, f.k_head, d), _at("v_head", v_head, dt, f.k_head, d),
            ctypes.byref(_mod(f, mod, d)), _at("o_head", o_head, dt, f.q_head, d),
            _at("lse", lse, torch.float32, f.lse, d), w, nw)


def ulysses_attn_bwd_mod(prob, q_head, k_head, v_head, o_head, lse, do_seq, mod: ScoreMod, dq_seq, dk_seq, dv_seq, ws,
                         stream=None):
    """The backward of ulysses_attn_fwd_mod (phase-1 workspace)."""
    f = _facts(prob)
    dt, d = f.dtype, _device(q_head)
    w, nw = _bytes("ws", ws, d)
    _launch("ulysses_attn_bwd_mod", d, stream, f.ref, _at("q_head", q_head, dt, f.q_head, d),
            _at("k_head", k_head, dt, f.k_head, d), _at("v_head", v_head, dt, f.k_head, d),
            _at("o_head", o_head, dt, f.q_head, d), _at("lse", lse, torch.float32, f.lse, d),
            _at("do_seq", do_seq, dt, f.q_seq, d), ctypes.byref(_mod(f, mod, d)),
            _at("dq_seq", dq_seq, dt, f.q_seq, d), _at("dk_seq", dk_seq, dt, f.k_seq, d),
            _at("dv_seq", dv_seq, dt, f.k_seq, d), w, nw)


# ---------------------------------------------------------------- buffers

def seq_layout(x: torch.Tensor, P: int) -> torch.Tensor:
    """Global [B, S, ...] -> rank-major sequence shards [P, B, S/P, ...]
    (rank r holds tokens [r*S/P, (r+1)*S/P)); a layout copy, no arithmetic."""
    B, S = x.shape[0], x.shape[1]
    return x.reshape(B, P, S // P, *x.shape[2:]).transpose(0, 1).contiguous()


class Buffers:
    """Device buffers for one problem: sequence-sharded inputs, head-sharded
    intermediates, outputs and the workspace (allocated by torch, owned by
    the caller, as the C ABI requires)."""

    def __init__(self, prob: Problem, device="cuda", backward: bool = False, fused: bool = False,
                 ds: bool = False):
        dt, p = prob.torch_dtype, prob
        D = p.head_dim
        e = lambda *s, d=dt: torch.empty(*s, dtype=d, device=device)
        self.q_seq = e(p.P, p.B, p.Sl, p.n_head, D)
        self.k_seq = e(p.P, p.B, p.Sl, p.n_kv_head, D)
        self.v_seq = e(p.P, p.B, p.Sl, p.n_kv_head, D)
        self.q_head = e(p.P, p.B, p.Cs, p.hp, D)
        self.k_head = e(p.P, p.B, p.Cs, p.kvp, D)
        self.v_head = e(p.P, p.B, p.Cs, p.kvp, D)
        self.o_head = e(p.P, p.B, p.Cs, p.hp, D)
        self.lse = e(p.P, p.B, p.hp, p.Cs, d=torch.float32)
        self.o_seq = e(p.P, p.B, p.Sl, p.n_head * D)
        if backward:
            self.do_seq = e(p.P, p.B, p.Sl, p.n_head * D)
            self.dq_seq = e(p.P, p.B, p.Sl, p.n_head, D)
            self.dk_seq = e(p.P, p.B, p.Sl, p.n_kv_head, D)
            self.dv_seq = e(p.P, p.B, p.Sl, p.n_kv_head, D)
            # gradients between the attention's backward and the norms'
            self.dqn_seq = e(p.P, p.B, p.Sl, p.n_head, D)
            self.dkn_seq = e(p.P, p.B, p.Sl, p.n_kv_head, D)
        # phase 2 (the fused backward's dQ accumulator) and phase 3 (the dS
        # store) when asked for
        phases = [1] + [2] * fused + [3] * ds if backward else [0]
        nbytes = max(ulysses_workspace_bytes(prob, ph) for ph in phases)
        if nbytes == 0:
            raise UlyssesError("ulysses_workspace_bytes", ulysses_validate(prob))
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.prob = prob

    def forward(self, stream=None):
        p = self.prob
        ulysses_pack_qkv(p, self.q_seq, self.k_seq, self.v_seq, self.q_head, self.k_head,
                         self.v_head, self.ws, stream)
        ulysses_attn_fwd(p, self.q_head, self.k_head, self.v_head, self.o_head, self.lse, self.ws,
                         stream)
        ulysses_unpack_out(p, self.o_head, self.o_seq, stream)

    def backward(self, stream=None):
        ulysses_attn_bwd(self.prob, self.q_head, self.k_head, self.v_head, self.o_head, self.lse,
                         self.do_seq, self.dq_seq, self.dk_seq, self.dv_seq, self.ws, stream)

    def forward_mod(self, mod: ScoreMod, norm=None, stream=None):
        """The forward with modified scores; norm: None, or (q_weight, k_weight,
        eps) of the query/key norms.  The norms' pack reads mod's mask too and
        writes zeros for padding, whatever it holds; without norms padding is
        packed as it is, and v_seq has to be finite there (for backward_mod q_seq
        and k_seq, too)."""
        p = self.prob
        if norm is None:
            ulysses_pack_qkv(p, self.q_seq, self.k_seq, self.v_seq, self.q_head, self.k_head, self.v_head, self.ws,
                             stream)
        else:
            ulysses_qk_norm_pack(p, self.q_seq, self.k_seq, self.v_seq, *norm, mod.mask, self.q_head, self.k_head,
                                 self.v_head, self.ws, stream)
        ulysses_attn_fwd_mod(p, self.q_head, self.k_head, self.v_head, mod, self.o_head, self.lse, self.ws, stream)
        ulysses_unpack_out(p, self.o_head, self.o_seq, stream)

    def backward_mod(self, mod: ScoreMod, norm=None, dnorm=None, stream=None):
        """The backward of forward_mod; with norm, the gradients of the norms'
        inputs end up in dq_seq and dk_seq too and those of the weights in
        dnorm = (dq_weight, dk_weight), float32 or None."""
        p = self.prob
        dq, dk = (self.dq_seq, self.dk_seq) if norm is None else (self.dqn_seq, self.dkn_seq)
        ulysses_attn_bwd_mod(p, self.q_head, self.k_head, self.v_head, self.o_head, self.lse, self.do_seq, mod, dq, dk,
                             self.dv_seq, self.ws, stream)
        if norm is not None:
            ulysses_qk_norm_bwd(p, self.q_seq, self.k_seq, *norm, dq, dk, self.dq_seq, self.dk_seq,
                                *(dnorm or (None, None)), self.ws, mod.mask, stream)

    def backward_fused(self, stream=None):
        ulysses_attn_bwd_fused(self.prob, self.q_head, self.k_head, self.v_head, self.o_head, self.lse,
                               self.do_seq, self.dq_seq, self.dk_seq, self.dv_seq, self.ws, stream)

    def backward_ds(self, stream=None):
        ulysses_attn_bwd_ds(self.prob, self.q_head, self.k_head, self.v_head, self.o_head, self.lse,
                            self.do_seq, self.dq_seq, self.dk_seq, self.dv_seq, self.ws, stream)
