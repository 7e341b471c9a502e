"""Padding that holds anything, for the attention with modified scores called by
itself: NaN and infinities in q and k of tokens that no row sees change nothing
for the others, whatever form of tanh their scores take."""
import dataclasses

import pytest
import torch

import modref as R
from test_gpu_qk_norm import plan_of
from test_gpu_score_mod import Case, forward, setup, workspace
from ulysses_sequence_attention_seq_gb300 import binding as U

pytestmark = pytest.mark.gpu

# Lengths of documents and (negative) of padding between them: the padding
# starts and ends at every offset within four neighbouring keys.
RUNS = [37, -1, 26, -6, 59, -2, 21, -9, 130, -3, 5, -17, 35, -41, 1, -1]

CASES = [  # scores past 0.6 of the cap (the exponential form) and well within it
    Case(cap=20.0, sigma=6.0), Case(cap=20.0, sigma=6.0, D=128, causal=False), Case(cap=20.0, sigma=1.0),
    Case(cap=90.0, sigma=12.0, D=128), Case(cap=90.0, sigma=12.0, causal=False), Case(cap=90.0, sigma=12.0, bias=True),
    Case(cap=20.0, sigma=6.0, bias=True, D=128, causal=False), Case(bias=True), Case(D=128),
    Case(dt="fp32", cap=20.0, sigma=6.0), Case(dt="fp32", D=128, cap=20.0, sigma=6.0, causal=False),
    Case(dt="fp32", D=32, cap=10.0, sigma=4.0, bias=True),
]


@pytest.mark.parametrize("c", CASES, ids=str)
def test_padding_may_hold_anything(c):
    """Bounds: modref.py's (float32: as test_forward_float32)."""
    S = sum(abs(n) for n in RUNS)
    c = dataclasses.replace(c, S=S, H=4, KV=2, B=2)
    prob, x, _, slopes, _ = setup(c)
    row = torch.cat([torch.full((abs(n),), -1 if n < 0 else i, dtype=torch.int32) for i, n in enumerate(RUNS)])
    doc = torch.stack([row, row.flip(0)])
    see = R.seen(c.B, S, c.causal, doc)
    dead = doc < 0
    for n in "qk":
        x[n][dead] = 0.0
    d = {n: x[n].to(R.F64) for n in x}
    val, bnd = R.attention_bounds(d["q"], d["k"], d["v"], None, see, prob.scale(), c.cap, slopes)
    if c.dt == "fp32":
        A, _ = R.attention(d["q"], d["k"], d["v"].abs(), see, prob.scale(), c.cap, slopes)
        e = 2 * bnd["lse"].transpose(1, 2)[..., None] + 2 * S * R.U32
        e = torch.where(torch.isfinite(e), e, torch.zeros_like(e))
        bnd["o"] = e * A + R.U32 * val["o"].abs() + 1e-30
    mod = U.ScoreMod(softcap=c.cap, slopes=None if slopes is None else slopes.cuda(), mask=plan_of(prob, doc))
    ws = workspace(prob, 0)
    fills = [float("nan"), float("inf"), -float("inf")]
    for k_fill in fills:
        for n, fill in (("q", fills[0]), ("k", k_fill)):
            x[n][dead] = fill
        _, o, lse = forward(prob, x, mod, ws)
        R.assert_within(R.from_head(o.cpu()), val["o"], bnd["o"], f"o, k {k_fill}")
        R.assert_within(R.lse_from_head(lse.cpu()), val["lse"], bnd["lse"], f"lse, k {k_fill}")


def test_plans_of_other_sizes_are_told_apart():
    """A plan says which sizes it is of in full.  (257, 1024) and (1, 125184) are two
    that a 32-bit hash of batch, length and flag took for one; the buffer has room
    for both."""
    small = dict(n_head=1, n_kv_head=1, head_dim=64, hidden=64, P=1, use_rope=False)
    made, used = U.Problem(B=257, S=1024, **small), U.Problem(B=1, S=125184, **small)
    n = max(U.ulysses_mask_bytes(made), U.ulysses_mask_bytes(used))
    plan = torch.empty(n, dtype=torch.uint8, device="cuda")
    U.ulysses_mask_build(made, None, None, 100, plan)
    ws = workspace(used, 1)
    q, k, v, o = (torch.zeros(1, 1, used.S, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    lse = torch.zeros(1, 1, 1, used.S, device="cuda")
    g = [torch.full_like(q, 5.0) for _ in range(3)]
    o.fill_(3.0), lse.fill_(3.0)
    mod = U.ScoreMod(mask=plan)
    U.ulysses_qk_norm_pack(used, q, k, v, None, None, 1e-6, plan, *g, ws)
    assert U.ulysses_read_status(ws) == U.STATUS_MASK and all((t == 5.0).all() for t in g)
    U.ulysses_workspace_init(used, ws)
    U.ulysses_attn_fwd_mod(used, q, k, v, mod, o, lse, ws)
    assert U.ulysses_read_status(ws) == U.STATUS_MASK and (o == 3.0).all() and (lse == 3.0).all()
    U.ulysses_workspace_init(used, ws)
    U.ulysses_attn_bwd_mod(used, q, k, v, o, lse, torch.zeros(1, 1, used.S, 64, dtype=torch.bfloat16, device="cuda"),
                           mod, *g, ws)
    assert U.ulysses_read_status(ws) == U.STATUS_MASK and all((t == 5.0).all() for t in g)
    U.ulysses_workspace_init(used, ws)
    U.ulysses_mask_build(used, None, None, 100, plan)      # and the same buffer with a plan of its own
    U.ulysses_attn_fwd_mod(used, q, k, v, mod, o, lse, ws)
    assert U.ulysses_read_status(ws) == 0 and (o == 0.0).all()
