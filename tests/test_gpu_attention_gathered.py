"""Prefill over pages that are gathered row by row: hidden non-finite values in every piece of a partly seen V tile."""
import pytest
import torch

from attn_testutil import Case, check

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,page", [(128, 24), (128, 1), (128, 100), (64, 24), (64, 5)])
def test_nonfinite_values_from_some_token_on(D, page, dtype):
    """From a token on every element of V is NaN or an infinity: whatever tile and piece it lies in, the rows before it
    are right and the rows from it on are not finite."""
    from quantized_gemm_error_gb300 import spear
    n, B = 400, 24
    hot = [16 * b + b % 16 for b in range(1, B + 1)]                # 17, 34, ... 392: every place in a warp's rows
    c = Case([n] * B, [n] * B, Hq=2, Hkv=1, D=D, page=page, dtype=dtype, seed=page)
    ref = c.reference()
    for b in range(B):
        for j in range(hot[b], n):
            c.v[c.table[b, j // page].item(), :, j % page] = (float("nan"), float("inf"), float("-inf"))[(b + j) % 3]
    cache, first = c.cache(), None
    sees = torch.cat([torch.arange(n) >= h for h in hot])
    for _ in range(10):
        out = spear.spear_attn_prefill(c.q_dev, cache, c.table, c.seq_lens, c.starts, scale=c.scale)
        torch.cuda.synchronize()
        assert spear.spear_get_device_status() == 0
        got = out.double().cpu()
        assert not torch.isfinite(got[sees]).any()
        got[sees] = ref[0][sees]
        check(got, None, ref, f"{D} page {page}")
        first = got if first is None else first
        assert torch.equal(got, first)


@pytest.mark.parametrize("window,sinks", [(60, 0), (130, 3)])
@pytest.mark.parametrize("D,page", [(128, 24), (128, 7), (64, 24)])
def test_nonfinite_values_behind_a_window(D, page, window, sinks):
    """The same up to a token: rows whose window is past it are right."""
    from quantized_gemm_error_gb300 import spear
    n = 500
    hot = [40, 128, 171, 255]
    c = Case([n] * 4, [n] * 4, Hq=2, Hkv=1, D=D, page=page, seed=page)
    ref = c.reference(window, sinks)
    for b in range(4):
        for j in range(sinks, hot[b]):
            c.v[c.table[b, j // page].item(), :, j % page] = float("nan")
    sees = torch.cat([(torch.arange(n) >= sinks) & (torch.arange(n) - window + 1 < h) for h in hot])
    for _ in range(10):
        out = spear.spear_attn_prefill(c.q_dev, c.cache(), c.table, c.seq_lens, c.starts, scale=c.scale, window=window,
                                       sinks=sinks)
        torch.cuda.synchronize()
        assert spear.spear_get_device_status() == 0
        got = out.double().cpu()
        assert not torch.isfinite(got[sees]).any()
        got[sees] = ref[0][sees]
        check(got, None, ref, f"{D} page {page} window {window}")
