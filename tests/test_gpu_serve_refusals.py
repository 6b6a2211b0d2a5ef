"""PagedServer refuses inputs and blocks that do not fit before anything is launched or counted."""
import pytest
import torch

from test_gpu_serve import _layer

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _block(D=64, q=256, k=128, v=128, o=None, width=512):
    from quantized_gemm_error_gb300.serve import AttentionBlock
    return AttentionBlock(_layer(width, q, 0), _layer(width, k, 1), _layer(width, v, 2), _layer(o or q, 512, 3), D)


def test_inputs_that_do_not_fit():
    from quantized_gemm_error_gb300 import spear
    from quantized_gemm_error_gb300.serve import PagedServer
    s = PagedServer([_block()], 8, 16, 4, 4, "cuda")
    x = torch.ones(6, 512, dtype=BF16, device="cuda")
    s.step(x[:3], [0], [3])
    torch.cuda.synchronize()
    before = [s.caches[0].k.clone(), s.caches[0].v.clone(), s.pool.snapshot()]
    wide = torch.ones(6, 1024, dtype=BF16, device="cuda")
    for bad in (x.float(), x.half(), x[:, :256].contiguous(), x[:, :, None], x.cpu(), wide[:, ::2]):
        with pytest.raises(ValueError):
            s.step(bad, [0, 1], [2, 4])
        torch.cuda.synchronize()
        assert spear.spear_get_device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(before, [s.caches[0].k, s.caches[0].v, s.pool.state]))
        assert s.count.lens == [3, 0, 0, 0]
    s.step(x, [0, 1], [2, 4])
    torch.cuda.synchronize()
    assert s.pool.seq_lens.tolist() == s.count.lens == [5, 4, 0, 0]


def test_blocks_that_do_not_fit():
    from quantized_gemm_error_gb300.serve import PagedServer
    for bad in (dict(q=384, k=256, v=256), dict(v=256), dict(o=512), dict(D=128, k=192, v=192),
                dict(D=128, q=320, o=384)):
        with pytest.raises(ValueError, match="block 1"):
            PagedServer([_block(), _block(**bad)], 8, 16, 4, 4, "cuda")
    with pytest.raises(ValueError, match="block 1"):
        PagedServer([_block(), _block(width=1024)], 8, 16, 4, 4, "cuda")
