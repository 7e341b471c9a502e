"""A distance bias over the Ulysses x ring hybrid: the forward then walks key
tiles from the last to the first, back over ring chunks, and slopes go by the
member's heads."""
import pytest

import test_gpu_score_mod as base
from test_gpu_score_mod import Case, check_forward, forward, setup, workspace

pytestmark = base.pytestmark

CASES = [  # chunks of 256 to 512 tokens: several tiles each
    Case(P=4, S=1024, H=4, KV=4, ring=2, bias=True), Case(P=4, S=1024, H=4, KV=2, ring=4, bias=True, D=128),
    Case(P=4, S=1024, H=4, KV=2, ring=2, bias=True, causal=False, B=2),
    Case(P=4, S=1024, H=8, KV=2, ring=4, bias=True, causal=False, cap=15.0, sigma=3.0),
    Case(P=8, S=2048, H=4, KV=1, ring=4, bias=True, cap=30.0, D=128, rope=True),
    # a window and documents: hulls that start and end inside chunks
    Case(P=4, S=1024, H=4, KV=4, ring=4, bias=True, window=300),
    Case(P=4, S=1536, H=4, KV=2, ring=4, bias=True, window=200, mean=400, pad=True, cap=20.0, D=128),
    Case(P=4, S=1024, H=4, KV=2, ring=2, bias=True, prefix=True, mean=300, rope=True),
]


@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward(c):
    prob, x, see, slopes, mod = setup(c)
    _, o, lse = forward(prob, x, mod, workspace(prob, 0))
    check_forward(c, prob, x, see, slopes, o, lse)


@pytest.mark.parametrize("c", CASES, ids=str)
def test_backward(c):
    base.test_backward(c)
