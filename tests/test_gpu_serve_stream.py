"""PagedServer on a stream of its own, with work ahead of its calls on either stream and allocations between them, against
the same steps on the current stream, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
STEPS = [("step", [0, 1, 5], [70, 33, 1]), ("step", [0, 1, 5], [1, 40, 17]), ("step", [0, 1, 5], [1, 1, 1]),
         ("fork", [0, 0, 1], [2, 3, 6]), ("step", [0, 2, 3, 6, 5], [1, 1, 1, 1, 1]), ("finish", [0, 5]), ("compact",),
         ("step", [2, 3, 1, 6], [1, 1, 1, 1]), ("step", [4, 0, 3], [100, 5, 1]), ("step", [0, 1, 2, 3, 4, 6], [1] * 6),
         ("finish", [1, 4]), ("compact",), ("step", [1, 2], [9, 1])]
WAIT = 4_000_000                                             # clocks of a kernel that does nothing (2 ms)


def _blocks():
    from quantized_gemm_error_gb300.serve import AttentionBlock
    from test_gpu_serve import _layer
    blocks = []
    for i, (hq, hkv, D) in enumerate([(8, 2, 64), (4, 4, 128)]):
        mk = lambda j, K, N: _layer(K, N, 100 * i + j, 16)
        blocks.append(AttentionBlock(mk(0, 512, hq * D), mk(1, 512, hkv * D), mk(2, 512, hkv * D), mk(3, hq * D, 512), D))
    return blocks


def _run(blocks, stream, busy):
    """Outputs (copied on the caller's stream) and the pool's state after each call."""
    from quantized_gemm_error_gb300.serve import PagedServer
    g = torch.Generator("cuda").manual_seed(1)
    got, litter = [], []
    s = PagedServer(blocks, 200, 16, 8, 40, "cuda", stream)
    for name, *args in STEPS:
        if busy and stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(WAIT)                      # the server's stream is behind the caller's
        if busy:
            torch.cuda._sleep(WAIT // 2)                     # and x is made late on the caller's
        if name == "step":
            x = torch.randn(sum(args[1]), 512, generator=g, device="cuda").to(BF16)
            outs = s.step(x, *args)
            del x
            got.append([y.clone() for y in outs])
            del outs
        else:
            getattr(s, name)(*args)
        # blocks of the sizes that the call gave back, overwritten at once on the caller's stream
        litter = [torch.full((n,), 7, dtype=torch.int32, device="cuda") for n in (1, 2, 3, 4, 5, 6, 7, 64, 512, 4096, 40000) * 3]
        del litter
        got.append([s.pool.snapshot()])
    torch.cuda.synchronize()
    # (what lies past the sequences' ends in their pages is stale, but the same)
    return got, [t for c in s.caches for t in (c.k, c.v)]


@pytest.mark.parametrize("busy", [False, True])
def test_a_side_stream_gives_the_same_bits(busy):
    from quantized_gemm_error_gb300 import spear
    blocks = _blocks()
    torch.cuda.synchronize()
    want, kv = _run(blocks, None, False)
    got, kv2 = _run(blocks, torch.cuda.Stream(), busy)
    assert spear.spear_get_device_status() == 0
    for a, b in zip(want, got):
        assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(torch.equal(a, b) for a, b in zip(kv, kv2))


def test_a_refused_step_leaves_the_streams_as_they_were():
    from quantized_gemm_error_gb300 import spear
    from quantized_gemm_error_gb300.serve import PagedServer, PoolFull
    s = PagedServer(_blocks(), 4, 16, 4, 8, "cuda", torch.cuda.Stream())
    here = torch.cuda.current_stream()
    x = torch.ones(70, 512, dtype=BF16, device="cuda")
    with pytest.raises(PoolFull):
        s.step(x, [0], [70])
    assert torch.cuda.current_stream() == here
    assert all(y.shape == (20, 512) for y in s.step(x[:20], [0], [20]))
    assert torch.cuda.current_stream() == here
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0


@pytest.mark.parametrize("side", [False, True])
def test_no_call_waits_for_the_gpu(side):
    """Synchronising calls raise meanwhile, and with a long kernel ahead on the stream all calls return before it ends."""
    from quantized_gemm_error_gb300 import spear
    from quantized_gemm_error_gb300.serve import PagedServer
    s = PagedServer(_blocks(), 200, 16, 8, 40, "cuda", torch.cuda.Stream() if side else None)
    x = torch.ones(80, 512, dtype=BF16, device="cuda")
    s.step(x[:40], [0, 7], [39, 1])                          # (what a first call sets up)
    s.step(x[:2], [0, 7], [1, 1])
    s.fork([0], [1])
    s.finish([1, 7])
    s.compact()
    torch.cuda.synchronize()
    begun = torch.cuda.Event()
    torch.cuda.set_sync_debug_mode("error")
    try:
        torch.cuda._sleep(400_000_000)                       # 0.2 s
        begun.record()
        s.step(x, [2, 3], [70, 10])
        s.step(x[:2], [2, 3], [1, 1])
        s.fork([2], [4])
        s.finish([3])
        s.compact()
        s.step(x[:2], [2, 4], [1, 1])
        waited = begun.query()
    finally:
        torch.cuda.set_sync_debug_mode("default")
    assert not waited
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    assert s.pool.seq_lens.tolist() == s.count.lens


def test_empty_calls():
    from quantized_gemm_error_gb300 import spear
    from quantized_gemm_error_gb300.serve import PagedServer
    s = PagedServer(_blocks(), 20, 16, 4, 8, "cuda")
    x = torch.ones(3, 512, dtype=BF16, device="cuda")
    s.step(x, [0, 1], [3, 0])
    s.finish([])
    s.fork([], [])
    assert [tuple(y.shape) for y in s.step(x[:0], [0], [0])] == [(0, 512)] * 2
    assert [tuple(y.shape) for y in s.step(x[:0], [], [])] == [(0, 512)] * 2
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    assert s.pool.seq_lens.tolist() == [3, 0, 0, 0]
