"""The bounds of the delta rule's GPU tests in the 2-norm, on the CPU: the form in
blocks with operands of the terms that the kernels take keeps them, and one
operand of fewer terms does not."""

import numpy as np
import pytest

from delta_terms import F32, OPERANDS, bf16, delta_in_terms, rms_bounds
from oracle import layer_oracle as ref

# fp32 io: what three terms and fp32 sums leave of y and of the state (delta_terms)
FP32_OFF = 2.0 ** -20
BF16_TERMS = {o: 1 if o in ("K", "Q", "S of y", "M", "U of y", "K of the state") else 2 for o in OPERANDS}


def head(L, P, N, keys=None, low=0.0, high=2.0, decay=0.0, length=0.98, to=F32, seed=0):
    """Inputs of a head, in the type's values; `keys` of them, drawn again and again."""
    rng = np.random.default_rng(seed)
    unit = lambda v: v / np.linalg.norm(v, axis=1, keepdims=True) * length  # noqa: E731
    x, k, q = to(rng.standard_normal((L, P))), to(unit(rng.standard_normal((keys or L, N)))), to(unit(rng.standard_normal((L, N))))
    if keys:
        k = k[rng.integers(0, keys, L)]
    beta = to((low + (high - low) * rng.random(L)) * (0.98 / length) ** 2)
    a = np.exp2(-decay * rng.random(L)).astype(F32)
    return [v.astype(np.float64) for v in (x, a, beta, k, q)] + [0.5, rng.standard_normal((P, N)) * 0.5]


def off(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("N", [32, 64, 128])
def test_one_operand_of_two_terms_is_seen(N):
    """Without a decay, so that what one block leaves the next ones keep."""
    args = head(300, 24, N, seed=N)
    y, S = ref.delta_rule(*args)
    yt, St = delta_in_terms(*args, {})
    assert off(yt, y) < FP32_OFF / 2 and off(St, S) < FP32_OFF / 2
    for o in OPERANDS:
        yt, St = delta_in_terms(*args, {o: 2})
        assert off(yt, y) > 1.5 * FP32_OFF, o
        if o not in ("Q", "S of y", "M", "U of y"):
            assert off(St, S) > 1.5 * FP32_OFF, o


@pytest.mark.parametrize("keys,low,high", [(1, 0.9, 1.1), (1, 1.9, 2.0), (3, 1.9, 2.0), (None, 0.0, 2.0)])
@pytest.mark.parametrize("decay,length", [(0.0, 0.98), (0.05, 0.5)])
def test_bf16_operands_keep_their_bounds(keys, low, high, decay, length):
    args = head(200, 24, 64, keys, low, high, decay, length, bf16)
    y, S = ref.delta_rule(*args)
    yt, St = delta_in_terms(*args, BF16_TERMS)
    yb, Sb = rms_bounds(*args, fp32=False)
    assert np.linalg.norm(yt - y) < yb and np.linalg.norm(St - S) < Sb
    # one term of all that reaches a state is seen
    yt, St = delta_in_terms(*args, {o: 1 for o in OPERANDS})
    assert np.linalg.norm(St - S) > Sb
