"""Without a GPU: the refusals of the norm, mask and modified-attention entry
points (fake pointers, never dereferenced), the plan's size, the Python
layer's checks, and the float64 forms the GPU tests rely on (modref.py)
against differences and worked examples."""
import copy
import ctypes
import dataclasses
import os
import pickle

import pytest
import torch

import modref as R
from ulysses_sequence_attention_seq_gb300 import binding as U
from ulysses_sequence_attention_seq_gb300 import build as B

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(U.LIB_PATH):
        B.build()
    return U.lib()


def prob(**kw):
    base = dict(B=1, S=1024, hidden=4096, n_head=32, n_kv_head=8, head_dim=128, P=8)
    base.update(kw)
    return U.Problem(**base)


def far(n):
    return [(1 << 40) + i * (1 << 34) for i in range(n)]


def norm_pack(lib, p, a, eps=1e-6, mask=0, mask_bytes=0, ws=None):
    n = U.ulysses_workspace_bytes(p, 0) if ws is None else ws
    return lib.ulysses_qk_norm_pack(ctypes.byref(p.c()), *[vp(x) for x in a[:5]], eps, vp(mask), mask_bytes,
                                    *[vp(x) for x in a[5:9]], n, vp(0))


def test_norm_pack_refusals(lib):
    p = prob()
    a = far(9)  # q k v wq wk qh kh vh ws
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert norm_pack(lib, p, a, eps=eps) == -1
    for i in (0, 1, 2, 5, 6, 7):
        assert norm_pack(lib, p, a[:i] + [0] + a[i + 1:]) == -1, i
    assert norm_pack(lib, p, a[:8] + [0]) == -7
    assert norm_pack(lib, p, a, ws=256) == -7
    for i in range(9):
        assert norm_pack(lib, p, a[:i] + [a[i] + 8] + a[i + 1:]) == -5, i
    assert norm_pack(lib, p, a[:5] + [a[0]] + a[6:]) == -6                 # q_head over q_seq
    assert norm_pack(lib, p, a[:5] + [a[3] - 4096] + a[6:]) == -6          # q_head over a weight
    assert norm_pack(lib, p, a, mask=1 << 46, mask_bytes=U.ulysses_mask_bytes(p) - 256) == -7
    assert norm_pack(lib, p, a, mask=(1 << 46) + 4, mask_bytes=U.ulysses_mask_bytes(p)) == -5
    assert norm_pack(lib, prob(n_kv_head=3), a, ws=1 << 30) == -2


def norm_bwd(lib, p, a, eps=1e-6, ws=None):
    n = U.ulysses_workspace_bytes(p, 1) if ws is None else ws
    return lib.ulysses_qk_norm_bwd(ctypes.byref(p.c()), *[vp(x) for x in a[:4]], eps, vp(0), 0,
                                   *[vp(x) for x in a[4:11]], n, vp(0))


def test_norm_backward_refusals(lib):
    p = prob()
    a = far(11)  # q k wq wk dqn dkn dq dk dwq dwk ws
    assert norm_bwd(lib, p, a, eps=0.0) == -1
    for i in (0, 1, 4, 5, 6, 7):
        assert norm_bwd(lib, p, a[:i] + [0] + a[i + 1:]) == -1, i
    assert norm_bwd(lib, p, a, ws=U.ulysses_workspace_bytes(p, 1) - 256) == -7
    assert norm_bwd(lib, p, a[:6] + [a[4]] + a[7:]) == -6                  # in place: refused
    assert norm_bwd(lib, p, a[:8] + [a[9], a[9]] + a[10:]) == -6           # both weight gradients in one place
    assert norm_bwd(lib, p, a[:9] + [a[9] + 4] + a[10:]) == -5


def build(lib, p, doc=0, prefix=0, window=0, mask=1 << 46, n=None):
    n = U.ulysses_mask_bytes(p) if n is None else n
    return lib.ulysses_mask_build(ctypes.byref(p.c()), vp(doc), vp(prefix), window, vp(mask), n, vp(0))


def test_mask_refusals(lib):
    p = prob()
    assert build(lib, p, mask=0) == -1
    assert build(lib, p, window=-1) == -1
    assert build(lib, prob(causal=False), prefix=1 << 40) == -1
    assert build(lib, p, n=U.ulysses_mask_bytes(p) - 1) == -7
    assert build(lib, p, doc=(1 << 40) + 4) == -5
    assert build(lib, p, doc=(1 << 46) + 256) == -6
    big = prob(S=(1 << 22) + 8, n_head=8, n_kv_head=8, hidden=1024)
    assert U.ulysses_validate(big) == 0 and U.ulysses_mask_bytes(big) == 0
    assert build(lib, big, n=1 << 40) == -4
    wide = prob(B=65536, S=8)
    assert U.ulysses_mask_bytes(wide) == 0 and build(lib, wide, n=1 << 40) == -4
    assert U.ulysses_mask_bytes(prob(B=0)) == 0


def test_mask_bytes(lib):
    p = prob(S=1024, B=2)  # 8 tiles: intervals of rows and keys, hulls, ends, edges, counts, lists
    assert U.ulysses_mask_bytes(p) == 256 + 2 * (2 * 1024 * 8) + 2 * (2 * 8 * 16) + 256 + 256 + 256


def fwd(lib, p, a, mod, ws=None):
    n = U.ulysses_workspace_bytes(p, 0) if ws is None else ws
    return lib.ulysses_attn_fwd_mod(ctypes.byref(p.c()), *[vp(x) for x in a[:3]],
                                    None if mod is None else ctypes.byref(mod), *[vp(x) for x in a[3:6]], n, vp(0))


def bwd(lib, p, a, mod, ws=None):
    n = U.ulysses_workspace_bytes(p, 1) if ws is None else ws
    return lib.ulysses_attn_bwd_mod(ctypes.byref(p.c()), *[vp(x) for x in a[:6]],
                                    None if mod is None else ctypes.byref(mod), *[vp(x) for x in a[6:10]], n, vp(0))


def test_attention_refusals(lib):
    p = prob()
    a = far(10)
    C = U.CScoreMod
    nb = U.ulysses_mask_bytes(p)
    for call in (fwd, bwd):
        assert call(lib, p, a, None) == -1
        for cap in (-1.0, float("nan"), float("inf"), 1e-4, 2.0 ** 21):
            assert call(lib, p, a, C(cap, None, None, 0)) == -1, cap
        assert call(lib, p, a, C(0.0, (1 << 46) + 4, None, 0)) == -5
        assert call(lib, p, a, C(0.0, None, (1 << 46) + 8, nb)) == -5
        assert call(lib, p, a, C(0.0, None, 1 << 46, nb - 1)) == -7
        assert call(lib, p, a, C(0.0, None, 1 << 46, 0)) == -7
        assert call(lib, p, a, C(20.0, None, None, 0), ws=0) == -7
        assert call(lib, prob(head_dim=32, hidden=1024), a, C(20.0, None, None, 0), ws=1 << 40) == -4
    # outputs over the slopes or the plan
    assert fwd(lib, p, a, C(0.0, a[4], None, 0)) == -6
    assert fwd(lib, p, a, C(0.0, None, a[3], nb)) == -6
    assert bwd(lib, p, a, C(0.0, a[7], None, 0)) == -6
    assert bwd(lib, p, a, C(0.0, None, a[9], nb)) == -6
    # no float32 backward
    assert bwd(lib, prob(dtype=U.FP32), a, C(20.0, None, None, 0), ws=1 << 40) == -4


def test_python_layer_refuses_what_the_library_cannot_see():
    p = prob(S=64, n_head=8, n_kv_head=8, hidden=1024)
    t = torch.empty(8, 1, 8, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        U.ulysses_qk_norm_pack(p, t, t, t, None, None, 1e-6, None, t, t, t, t)
    with pytest.raises(ValueError, match="CUDA tensor"):
        U.ulysses_mask_build(p, None, None, 0, torch.empty(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        U.ulysses_attn_fwd_mod(p, t, t, t, U.ScoreMod(), t, t, t)
    with pytest.raises(U.UlyssesError):
        U.ulysses_attn_fwd_mod(prob(P=0), t, t, t, U.ScoreMod(), t, t, t)


# ------------------------------------------------------- the float64 forms

def test_intervals_by_hand():
    doc = [0, 0, 0, -1, 0, 0, 5, 5]
    assert R.intervals(8, True, doc) == [(0, 1), (0, 2), (0, 3), (0, 0), (4, 5), (4, 6), (6, 7), (6, 8)]
    assert R.intervals(8, False, doc) == [(0, 3)] * 3 + [(0, 0)] + [(4, 6)] * 2 + [(6, 8)] * 2
    assert R.intervals(4, True, None, [2, 2, 9, -1]) == [(0, 2), (0, 2), (0, 4), (0, 4)]
    assert R.intervals(4, True, None, None, 2) == [(0, 1), (0, 2), (1, 3), (2, 4)]


def test_reference_gradients_against_differences():
    """The formulas behind the bounds (attention_bounds) give the gradients of
    the forward, and the forward's central differences agree with both."""
    g = torch.Generator().manual_seed(0)
    B, S, H, KV, D = 1, 9, 4, 2, 8
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=R.F64)
    q, k, v, do = rnd(B, S, H, D) * 2, rnd(B, S, KV, D) * 2, rnd(B, S, KV, D), rnd(B, S, H, D)
    see = R.seen(B, S, True, torch.tensor([[0, 0, 0, 0, -1, 3, 3, 3, 3]]), torch.tensor([[2] * 9]))
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.0], dtype=R.F64)
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    f = lambda q, k, v: (R.attention(q, k, v, see, 0.35, 1.5, slopes)[0] * do).sum()
    auto = torch.autograd.grad(f(*leaves), leaves)
    val, _ = R.attention_bounds(q, k, v, do, see, 0.35, 1.5, slopes)
    for n, a in zip(("dq", "dk", "dv"), auto):
        assert torch.allclose(val[n], a, rtol=1e-10, atol=1e-12), n
    h = 1e-5
    for i, a in enumerate(auto):
        for _ in range(3):
            d = rnd(*a.shape)
            args = [[q, k, v], [q, k, v]]
            args[0][i], args[1][i] = (q, k, v)[i] + h * d, (q, k, v)[i] - h * d
            diff = (f(*args[0]) - f(*args[1])) / (2 * h)
            # central differences: h^2 times a third derivative of order 1e2
            assert abs(diff - (a * d).sum()) <= 1e-6 * (1 + abs(diff))


def test_layouts_round_trip():
    x = torch.arange(2 * 24 * 4 * 2).reshape(2, 24, 4, 2)
    assert torch.equal(R.from_seq(R.to_seq(x, 4)), x)
    assert torch.equal(R.from_head(R.to_head(x, 4)), x)
    assert torch.equal(R.from_head(R.to_head(x, 4, 2), 2), x)


def test_a_used_problem_copies_and_pickles(lib):
    p = prob(S=64, n_head=8, n_kv_head=8, hidden=1024)
    t = torch.empty(8, 1, 8, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        U.ulysses_attn_fwd_mod(p, t, t, t, U.ScoreMod(), t, t, t)   # (works out the problem's sizes, then refuses)
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p)), dataclasses.replace(p)):
        assert q == p and hash(q) == hash(p) and vars(q) == dataclasses.asdict(p)
        with pytest.raises(ValueError):
            U.ulysses_attn_fwd_mod(q, t, t, t, U.ScoreMod(), t, t, t)


def test_a_layer_step_makes_no_buffer(lib, monkeypatch):
    """Everything a step writes is there before it, made on the stream that made
    the rest: a block the allocator hands out in the middle of a step belongs to
    the current stream, and the step may run on another."""
    p = prob(B=1, S=16, hidden=1024, n_head=8, n_kv_head=8)
    b = U.Buffers(p, device="cpu", backward=True)
    calls = []
    for name in ("ulysses_pack_qkv", "ulysses_qk_norm_pack", "ulysses_attn_fwd_mod", "ulysses_unpack_out",
                 "ulysses_attn_bwd_mod", "ulysses_qk_norm_bwd"):
        monkeypatch.setattr(U, name, lambda *a, name=name: calls.append((name, a)))
    for name in ("empty", "empty_like", "zeros", "zeros_like"):
        monkeypatch.setattr(torch, name, lambda *a, **k: pytest.fail("a tensor is made"))
    norm, stream = (None, None, 1e-6), object()
    b.forward_mod(U.ScoreMod(), norm, stream)
    b.backward_mod(U.ScoreMod(), norm, None, stream)
    assert [c[0] for c in calls] == ["ulysses_qk_norm_pack", "ulysses_attn_fwd_mod", "ulysses_unpack_out",
                                     "ulysses_attn_bwd_mod", "ulysses_qk_norm_bwd"]
    assert all(c[1][-1] is stream for c in calls)
    between = [t.data_ptr() for t in calls[3][1][8:10]]
    assert between == [t.data_ptr() for t in calls[4][1][6:8]]
    assert len({*between, b.dq_seq.data_ptr(), b.dk_seq.data_ptr()}) == 4


# ------------------------------------------------------------ read, not run

def test_barriers_behind_divergent_code_are_not_the_aligned_kind():
    """barrier.cluster's .aligned forms are defined only where a warp's lanes
    arrive together; the plan's kernel reaches its barriers from per-lane
    branches and a search whose length differs from lane to lane."""
    with open(os.path.join(B.CSRC, "mask.cu")) as f:
        asm = [line for line in f if "asm volatile" in line and "barrier.cluster" in line]
    assert asm and not any(".aligned" in line for line in asm)


@pytest.mark.parametrize("name", ["attn_fwd_mod_tc.cu", "attn_bwd_mod_tc.cu", "attn_fwd_mod_simt.cu"])
def test_reads_of_the_plan_ask_in_a_checked_build(name):
    """Entries of the plan, and slopes, are read behind in_range, there or in the
    helpers of mask.cuh and score_mod.cuh."""
    with open(os.path.join(B.CSRC, name)) as f:
        lines = f.read().split("\n")
    for i, line in enumerate(lines):
        if "__ldg(" in line and ("mask." in line or "slopes" in line or "list" in line or "__ldg(tl" in line):
            assert "in_range" in " ".join(lines[max(0, i - 1):i + 1]), f"{name}:{i + 1}"
