"""Values near the end of the type's range: an output is an average of them, and no sum on the way may overflow (as
long as the sum of a row's |v| does not pass fp32's range, 2^128)."""
import math

import pytest
import torch

from attn_testutil import Case, check

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def _scaled(dtype, D, growth, lens, new):
    """V times 2^114 (fp16: 2^13); the score of the key in the middle is `growth` nats above the first tiles'."""
    c = Case(lens, new, Hq=8, Hkv=8, D=D, page=16, dtype=dtype, seed=7, spread=0.2)
    big = 2.0 ** (114 if dtype is BF16 else 13)
    c.v *= big
    c.V = [v * big for v in c.V]
    c.q[:, :, 0] = math.sqrt(D)
    c.q_dev = c.q.cuda()
    for b, n in enumerate(lens):
        c.K[b][:, :, 0] = 0.0
        c.K[b][n // 2, :, 0] = growth
        pages = c.table[b, :-(-n // 16)].long()
        rows = torch.zeros(len(pages) * 16, 8, dtype=dtype)
        rows[:n] = c.K[b][:, :, 0]
        c.k[pages, :, :, 0] = rows.view(-1, 16, 8).transpose(1, 2).cuda()
    return c


@pytest.mark.parametrize("growth", [0.0, 9.5, 30.0])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("prefill", [False, True])
def test_large_values(prefill, dtype, D, growth):
    from quantized_gemm_error_gb300 import spear
    lens = [400] * 6 if prefill else [300] * 20              # (prefill: enough that items are not all split into tiles)
    c = _scaled(dtype, D, growth, lens, lens if prefill else None)
    lse = torch.empty(c.q_dev.shape[:2], device="cuda")
    if prefill:
        out = spear.spear_attn_prefill(c.q_dev, c.cache(), c.table, c.seq_lens, c.starts, lse=lse)
    else:
        out = spear.spear_attn_decode(c.q_dev, c.cache(), c.table, c.seq_lens, lse=lse)
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    check(out, lse, c.reference(), f"{'prefill' if prefill else 'decode'} {dtype} {D} {growth}")
