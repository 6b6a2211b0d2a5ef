"""Arguments at the ends of their 32 bits, and past them."""
import pytest
import torch

from attn_testutil import Case, check

pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1


def _run(c, prefill, **kw):
    from quantized_gemm_error_gb300 import spear
    if prefill:
        out = spear.spear_attn_prefill(c.q_dev, c.cache(), c.table, c.seq_lens, c.starts, **kw)
    else:
        out = spear.spear_attn_decode(c.q_dev, c.cache(), c.table, c.seq_lens, **kw)
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefill", [False, True])
def test_windows_and_sinks_past_every_key(prefill, D):
    c = Case([300, 5], [200, 9] if prefill else None, Hq=4, Hkv=2, D=D)      # (four tokens before position 0 see nothing)
    for window, sinks in ((TOP, 0), (TOP, TOP), (10, TOP), (299, 1), (300, 1)):
        check(_run(c, prefill, window=window, sinks=sinks), None, c.reference(window, sinks), f"{window} {sinks}")


@pytest.mark.parametrize("prefill", [False, True])
def test_numbers_that_do_not_fit_are_refused(prefill):
    from quantized_gemm_error_gb300 import spear
    c = Case([300], Hq=2, Hkv=1, D=64)
    for kw in (dict(window=TOP + 1), dict(window=2 ** 32), dict(window=2 ** 32 + 10), dict(window=10, sinks=2 ** 32),
               dict(window=10, sinks=2 ** 40 + 3),
               dict(window=-2 ** 32), dict(window=10, sinks=-2 ** 32)):
        with pytest.raises(ValueError, match="32-bit"):
            _run(c, prefill, **kw)
    for kw in (dict(window=-1), dict(sinks=-1), dict(window=-2 ** 31)):
        with pytest.raises(spear.SpearError):
            _run(c, prefill, **kw)
