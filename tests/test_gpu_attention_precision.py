"""What the chunks' products keep of numbers that cancel: three rows of a sequence whose last value
of out is 2^-16 of the terms it is made of, so that it shows what its own type would hide."""
import pytest
import torch

import selective_state_update_ssu_amd as ssu
from test_gpu_layer import Draw

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16
K, V, HEADS, NSEQ = 8, 64, 8, 40


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("io", [BF16, F16])
def test_products_of_rows_keep_what_cancels(io, delta):
    """Each key has two components of its own, so that keys are orthogonal (R is beta v, one rounding),
    and the second ones are so small that the two products of a score add up without one, to more bits
    than two bf16 parts hold. No decay. v of the second and third row take away what the rows
    before them give. Error of the sum: as many matrix instructions as there are pairs of parts (P and R
    in three, of v itself one or two: 3 and 5, with beta 6), each up to four additions that are off by a
    step of fp32, 2 u; parts left out and the rounding of beta v 2 u; and half a step of out."""
    d = Draw(6)
    rows = 3 * NSEQ
    q, k = (torch.zeros(rows, HEADS, K) for _ in range(2))
    for j in range(3):
        k[j::3, :, 2 * j] = d.uniform(1.0, 2.0, NSEQ, HEADS)
        k[j::3, :, 2 * j + 1] = d.uniform(1.0, 2.0, NSEQ, HEADS)
        q[2::3, :, 2 * j] = d.uniform(1.0, 2.0, NSEQ, HEADS)
        q[2::3, :, 2 * j + 1] = d.uniform(1.0, 2.0, NSEQ, HEADS) * 2.0 ** -7
    q, k = (x.to(BF16).to(io) for x in (q, k))  # numbers of 8 bits
    P = torch.stack([(q[2::3].double() * k[j::3].double()).sum(-1) for j in range(3)])[..., None]
    assert torch.equal(P, P.float().double()) and not torch.equal(P, P.to(BF16).double())
    beta = d.uniform(0.5, 1.0, rows, HEADS) if delta else None
    b = beta.double()[..., None] if delta else torch.ones(rows, HEADS, 1, dtype=torch.float64)
    v = torch.zeros(rows, HEADS, V, dtype=io)
    v[0::3] = d.uniform(1.0, 2.0, NSEQ, HEADS, V).to(io)
    for j in (1, 2):
        got = sum(P[i] * b[i::3] * v[i::3].double() for i in range(j))
        v[j::3] = (-got / (P[j] * b[j::3])).to(io)
    terms = [P[i] * b[i::3] * v[i::3].double() for i in range(3)]
    want, size = sum(terms), sum(t.abs() for t in terms)
    assert float((want.abs() / size).max()) < 2.0 ** -14
    products = 6 if delta else 3 if io == BF16 else 5
    bound = (products * 4 * 2 + 2) * 2.0 ** -24 * size + torch.finfo(io).eps / 2 * want.abs() + 2.0 ** -25
    out = ssu.linear_attention_varlen(
        torch.zeros(NSEQ, HEADS, V, K, device=DEV), q.to(DEV), k.to(DEV), v.to(DEV),
        torch.zeros(HEADS, device=DEV), torch.arange(0, rows + 1, 3, dtype=torch.int32, device=DEV),
        beta=beta.to(DEV) if delta else None)
    err = (out[2::3].double().cpu() - want).abs()
    assert bool((err <= bound).all())
