"""Shares of logits far below the largest, to the last bits of 32: expert_balance
and its gradient on the GPU against the definition in 64 bits.

A row holds the logit 0, one logit d and otherwise -inf, all of them numbers
of 16 bits: the difference d is exact, and what the row's sum adds are two powers
and zeros.  All choices are of d's expert.  To first order, in steps of u = 2**-24:
  a power is off by 2 ulp at most, 4 u of itself; the sum of two by 4 u and its
  rounding, 5 u; the quotient by a reciprocal and a product, 2 u: a share by 11 u;
  the loss E / n * share * c / C by three more products and quotients and that
  of E by n, 4 u: 15 u of itself;
  the gradient E / n * p * (1 - p), p <= 1/2: p by 11 u, 1 - p by 11 u of p and
  a rounding, of itself 12 u at most; its products by 4 u more and E / n, 5 u: 28 u.
One u on top for what is of second order.
"""

import pytest

import bmmc_index_transforms_gb300 as bm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
FAR = [-k / 2 for k in range(2, 161)]  # -1 .. -80


def _rows(E, dtype):
    x = torch.full((len(FAR), E), float("-inf"), dtype=dtype, device="cuda")
    x[:, 0] = 0
    x[:, E - 1] = torch.tensor(FAR, device="cuda").to(dtype)
    assert x[:, E - 1].double().tolist() == FAR
    p = torch.softmax(x.double(), 1)[:, E - 1]
    return x, torch.full((len(FAR), 1), E - 1, device="cuda"), p


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("E", [2, 61, 256, 512, 1000, 1500])
def test_loss_of_far_logits(E, dtype):
    x, ids, p = _rows(E, dtype)
    got = torch.stack([bm.expert_balance(x[t:t + 1], ids[t:t + 1])[0] for t in range(len(FAR))]).double()
    off = (got / (E * p) - 1).abs()
    assert float(off.max()) <= 16 * U32, (float(off.max()) / U32, FAR[int(off.argmax())])


@pytest.mark.parametrize("E", [2, 61, 256, 512, 1000, 1500])
def test_gradient_of_far_logits(E):
    x, ids, p = _rows(E, torch.float32)
    one = torch.ones((), device="cuda")
    _, counts = bm.expert_balance(x, ids)
    got = bm.expert_balance_backward(one, x, ids, counts).double()[:, E - 1]
    off = (got / (E / len(FAR) * p * (1 - p)) - 1).abs()
    assert float(off.max()) <= 29 * U32, (float(off.max()) / U32, FAR[int(off.argmax())])
