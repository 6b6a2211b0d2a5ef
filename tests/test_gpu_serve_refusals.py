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


@pytest.mark.parametrize("side", [False, True])
def test_a_pool_changed_from_outside_is_counted_anew(side):
    from quantized_gemm_error_gb300 import spear
    from quantized_gemm_error_gb300.serve import PagedServer, PoolFull
    s = PagedServer([_block()], 4, 16, 4, 4, "cuda", torch.cuda.Stream() if side else None)
    x = torch.ones(64, 512, dtype=BF16, device="cuda")
    s.step(x[:40], [0], [40])
    torch.cuda.synchronize()
    saved = s.pool.snapshot()
    s.step(x[:16], [1], [16])
    torch.cuda.synchronize()
    s.pool.restore(saved)                                    # the last step taken back
    torch.cuda.synchronize()
    with pytest.raises(PoolFull):
        s.step(x[:16], [2], [16])
    s.recount()
    assert s.count.lens == [40, 0, 0, 0] and s.count.free_pages == 1
    s.fork([0], [1])
    with pytest.raises(PoolFull):
        s.step(x[:9], [1], [9])
    s.step(x[:8], [1], [8])
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    assert s.pool.seq_lens.tolist() == s.count.lens == [40, 48, 0, 0]
    assert s.pool.refs.tolist() == [2, 2, 1, 1] and s.count.free_pages == 0
