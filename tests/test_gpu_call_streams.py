"""Calls on a stream that is not the current one: what they allocate must not be memory that the current stream has work
queued on, and results may be dropped while the current stream still reads them."""
import math

import pytest
import torch

from attn_testutil import Case

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
WAIT = 100_000_000                                         # clocks of a kernel that does nothing (50 ms)


def _calls():
    from quantized_gemm_error_gb300 import spear
    g = torch.Generator("cuda").manual_seed(0)
    W = torch.randn(512, 1024, generator=g, device="cuda") / 32
    q, s, z = spear.spear_pack_w4(W, 128, False)
    layer = spear.W4Layer(512, 1024, 128, False, q, s, z)
    xd, xp = (torch.randn(m, 1024, generator=g, device="cuda").to(BF16) for m in (7, 300))
    c, p = Case([700, 40], Hq=8, Hkv=2), Case([300, 90], [250, 90], Hq=4, Hkv=2)
    cc, cp = c.cache(), p.cache()
    return {
        "linear_decode": lambda st: spear.spear_linear_decode(layer, xd, stream=st),
        "linear_prefill": lambda st: spear.spear_linear_prefill(layer, xp, stream=st),
        "attn_decode": lambda st: spear.spear_attn_decode(c.q_dev, cc, c.table, c.seq_lens, stream=st),
        "attn_prefill": lambda st: spear.spear_attn_prefill(p.q_dev, cp, p.table, p.seq_lens, p.starts, stream=st),
        "pack_w4": lambda st: spear.spear_pack_w4(W, 128, False, stream=st)[0],
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["linear_decode", "linear_prefill", "attn_decode", "attn_prefill", "pack_w4"])
def test_results_do_not_land_in_memory_in_use(name, raw):
    from quantized_gemm_error_gb300 import spear
    call = _calls()[name]
    side = torch.cuda.Stream()
    st = side.cuda_stream if raw else side
    want = call(None)
    call(st)                                               # (the stream's workspace)
    torch.cuda.synchronize()
    fill = [torch.full_like(want, 3) for _ in range(8)]    # dropped below: blocks that fit the result
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    kept = [f.clone() for f in fill]                       # queued behind the wait
    del fill
    out = call(st)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all((k == 3).all() for k in kept)
    # dropped while the current stream still has to read it
    torch.cuda._sleep(WAIT)
    later = out.clone()
    del out
    for _ in range(3):
        call(st).zero_()
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(later, want)
    assert spear.spear_get_device_status() == 0


@pytest.mark.parametrize("name", ["linear_decode", "attn_decode", "attn_prefill"])
def test_workspaces_do_not_land_in_memory_in_use(name):
    from quantized_gemm_error_gb300 import spear
    call = _calls()[name]
    side = torch.cuda.Stream()
    spear.reset_default_workspaces()
    want = call(None)
    torch.cuda.synchronize()
    sizes = {w.numel() for w in spear._default_ws.values()}
    fill = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    kept = [f.clone() for f in fill]
    del fill
    out = call(side)                                       # its workspace is made (and zeroed) now
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all((k == 3).all() for k in kept)
    spear.reset_default_workspaces()
