"""fp16 attention where a row's largest probability belongs to a key whose value is zero (a sink): the output is made of
probabilities far below it.

Tolerance, relative, all terms of the output having one sign (u = 2^-11): the output's rounding u, p's u or, below fp16's
normal range, 2^-33 of the largest p, i.e. 2^-33 e^nats of p itself; fp32 errors of the scores (|s| (D + 4) 2^-23, the
terms of s having one sign), of the exponential 2^-20 and of the sums (n 2^-23), each twice."""
import math

import pytest
import torch

from attn_testutil import Case

pytestmark = pytest.mark.gpu
F16, U = torch.float16, 2.0 ** -11


def _sink_case(B, n, new, H, D, nats):
    """B sequences of n keys; key 0 has value 0 and a score `nats` above the others', whose values are 500 to 1500."""
    c = Case([n] * B, [new] * B, Hq=H, Hkv=H, D=D, page=16, dtype=F16, seed=1)
    g = torch.Generator().manual_seed(3)
    k = torch.zeros(n, D)
    k[0] = nats / math.sqrt(D)
    v = 1000.0 * (torch.rand(n, D, generator=g) + 0.5)
    v[0] = 0
    k, v = k.to(F16), v.to(F16)
    for b in range(B):
        for j in range(-(-n // 16)):
            m, page = min(16, n - 16 * j), c.table[b, j].item()
            c.k[page, :, :m], c.v[page, :, :m] = k[16 * j:16 * j + m].cuda(), v[16 * j:16 * j + m].cuda()
    c.q_dev.fill_(1.0)
    s = k.double().sum(-1) / math.sqrt(D)
    return c, s, v.double()


def _tolerance(s, n, D):
    c = s[0].item() * (D + 4) * 2.0 ** -23 + 2.0 ** -20 + n * 2.0 ** -23
    return 1.01 * (U + max(U, 2.0 ** -33 * math.exp(s[0].item())) + 2 * c)


@pytest.mark.parametrize("nats", [9, 12, 16, 17])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_keys_far_below_a_sink(D, nats):
    from quantized_gemm_error_gb300 import spear
    B, n, H = 128, 200, 16                       # items enough that a warp takes whole ones
    c, s, v = _sink_case(B, n, 1, H, D, nats)
    lse = torch.empty(B, H, device="cuda")
    out = spear.spear_attn_decode(c.q_dev, c.cache(), c.table, c.seq_lens, lse=lse)
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    ref = torch.softmax(s, 0) @ v
    err = ((out.double().cpu() - ref) / ref).abs().max().item()
    assert err <= _tolerance(s, n, D), (err, _tolerance(s, n, D))
    assert (lse.double().cpu() - torch.logsumexp(s, 0)).abs().max() <= 2 * _tolerance(s, n, D) - 2 * U


@pytest.mark.parametrize("nats", [9, 12, 16, 17])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_keys_far_below_a_sink(D, nats):
    from quantized_gemm_error_gb300 import spear
    B, n, H = 24, 300, 16
    c, s, v = _sink_case(B, n, n, H, D, nats)
    lse = torch.empty(B * n, H, device="cuda")
    out = spear.spear_attn_prefill(c.q_dev, c.cache(), c.table, c.seq_lens, c.starts, lse=lse)
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    w = torch.exp(s - s[0])
    ref = (torch.cumsum(w[:, None] * v, 0) / torch.cumsum(w, 0)[:, None]).view(1, n, 1, D)
    got = out.double().cpu().view(B, n, H, D)
    assert (got[:, 0] == 0).all()
    seen = ref[0, :, 0, 0] > 2.0 ** -14 * 2      # rows whose outputs are normal fp16 numbers
    assert seen.sum() > 100
    err = ((got - ref) / ref)[:, seen].abs().max().item()
    assert err <= _tolerance(s, n, D), (err, _tolerance(s, n, D))
    want = (s[0] + torch.cumsum(w, 0).log()).view(1, n, 1)
    assert (lse.double().cpu().view(B, n, H) - want).abs().max() <= 2 * _tolerance(s, n, D) - 2 * U


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_scores_that_keep_growing(D):
    """Each key's score is above the one before, by little or much: the running maximum moves often, and what was summed
    before it follows.  The tolerance of attn_testutil."""
    from attn_testutil import check
    from quantized_gemm_error_gb300 import spear
    for step in (0.02, 0.3, 3.0):
        c = Case([400, 270], [400, 30], Hq=2, Hkv=1, D=D, page=16, dtype=F16, seed=2)
        for b, n in ((0, 400), (1, 270)):
            k = (c.K[b] * 0.02).double()
            k[:, 0, 0] = torch.arange(n) * min(step, 600.0 / n)
            c.K[b] = k.to(F16)
            for j in range(n):
                c.k[c.table[b, j // 16].item(), :, j % 16] = c.K[b][j].cuda()
        c.q = c.q * 0.02
        c.q[:, :, 0] = math.sqrt(D)
        c.q = c.q.to(F16)
        c.q_dev = c.q.cuda()
        lse = torch.empty(430, 2, device="cuda")
        out = spear.spear_attn_prefill(c.q_dev, c.cache(), c.table, c.seq_lens, c.starts, lse=lse)
        torch.cuda.synchronize()
        assert spear.spear_get_device_status() == 0
        check(out, lse, c.reference(), f"step {step}")
