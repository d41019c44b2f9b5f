"""How exactly the tcgen05 scores take the logsumexp off.

Queries and keys are small whole numbers, so every q.k is exact in fp32, and one row alone has a logsumexp, so a score is one weight,
w = exp(tau s - lse).  s and lse / tau lie between 0.9 and 1 times a power of two, B.  The product takes s, the four terms of -lse / tau
and their sum at the size of B: each of the five is taken to be cut at a quarter of fp32's last place there, B 2^-24 (tensor cores add with a
few bits more than they give), and the terms are exact to 2^-32; what remains is small and exact in fp32.  So log2 w is within 1.25 B 2^-24 tau
log2(e), the scale's and the product's rounding within 2^-23 of |log2 w| together (2^-22 asked for), and the exponential and the sum
within 2^-21.
"""
import math

import pytest
import torch

import local_linear_attention_flashlla_gb300 as lla

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [40, 64])
@pytest.mark.parametrize("d,tau,B", [(128, 128 ** -0.5, 2.0 ** 14), (128, 0.037, 2.0 ** 14), (64, 0.1, 2.0 ** 13)])
def test_a_weight_is_as_exact_as_its_logit(lla_gpu, n, d, tau, B):
    gen = torch.Generator().manual_seed(0)
    L, page = 4096, 64
    q = torch.randint(8, 16, (n, 1, d), generator=gen).bfloat16()
    k = torch.randint(8, 16, (L, d), generator=gen).bfloat16()
    s = q[-1, 0].double() @ k.double().T
    tau = float(torch.tensor(tau, dtype=torch.float32))
    near = (s < B) & (s > 0.9 * B)
    assert int(near.sum()) > 20
    args = (k.reshape(L // page, 1, page, d).cuda(), torch.arange(L // page, dtype=torch.int32, device="cuda")[None],
            torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([L], dtype=torch.int32, device="cuda"))
    for _ in range(60):
        lse = torch.full((n, 1), -math.inf)
        lse[-1] = B * (0.985 + 0.0148 * torch.rand((), generator=gen)) * tau
        scores = torch.zeros(L // page, 1, page, device="cuda")
        lla.paged_weigh(q.cuda(), lse.cuda(), args[0], scores, *args[1:], tau, n, causal=False, decay=0.0)
        x = (tau * s - lse[-1].double()) / math.log(2)
        use = near & (x.abs() < 60)
        off = (torch.log2(scores.flatten().double().cpu()) - x).abs()
        tol = 1.25 * B * 2.0 ** -24 * tau / math.log(2) + 2.0 ** -22 * x.abs() + 2.0 ** -21
        assert (off <= tol)[use].all(), float((off / tol)[use].max())
    lla.lla_sync_status()
