"""A reservation that the pool refuses, and the calls after it: what is cached stays as it is."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _i(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(n, value):
    return torch.full((n, 2, 64), float(value), dtype=BF16, device="cuda")


def _full_pool():
    """Row 0 of two whole pages, row 1 forked from it (both pages shared), row 2 with the other two pages."""
    from quantized_gemm_error_gb300 import spear
    pool, cache = spear.PagePool(4, 4, 4, 4, "cuda"), spear.new_kv_cache(4, 4, 2, 64, "cuda")
    spear.spear_kv_reserve(pool, _i(0), _i(8))
    spear.spear_kv_append(cache, _rows(8, 1), _rows(8, 2), pool.block_table, pool.seq_lens, _i(0, 8), seq_ids=_i(0), pool=pool)
    spear.spear_kv_fork(pool, cache, _i(0), _i(1))
    spear.spear_kv_reserve(pool, _i(2), _i(8))
    spear.spear_kv_append(cache, _rows(8, 3), _rows(8, 4), pool.block_table, pool.seq_lens, _i(0, 8), seq_ids=_i(2), pool=pool)
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    assert pool.refs.tolist() == [2, 2, 1, 1] and (cache.k != 0).all()
    return pool, cache


def test_append_after_a_refused_reserve_writes_nothing():
    from quantized_gemm_error_gb300 import spear
    pool, cache = _full_pool()
    k, v, state = cache.k.clone(), cache.v.clone(), pool.snapshot()
    append = lambda row: spear.spear_kv_append(cache, _rows(2, 9), _rows(2, 9), pool.block_table, pool.seq_lens, _i(0, 2),
                                               seq_ids=_i(row), pool=pool)
    for row, tokens in ((1, 2), (2, 2), (0, 100), (7, 1)):     # no page free (two rows), too long for a row, no such row
        spear.spear_kv_reserve(pool, _i(row), _i(tokens))
        torch.cuda.synchronize()
        assert spear.spear_get_device_status() == 1
        append(min(row, 3))
        torch.cuda.synchronize()
        assert spear.spear_get_device_status() == 1
        assert torch.equal(cache.k, k) and torch.equal(cache.v, v) and torch.equal(pool.state, state)
    # other bookkeeping in between does not forget it
    spear.spear_kv_reserve(pool, _i(1), _i(2))
    spear.spear_kv_fork(pool, cache, _i(0), _i(3))
    spear.spear_kv_free(pool, _i(3))
    spear.spear_kv_compact(pool, cache)
    append(1)
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 1
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v) and torch.equal(pool.state, state)
    # and with room again all goes on
    spear.spear_kv_free(pool, _i(2))
    spear.spear_kv_reserve(pool, _i(1), _i(2))
    append(1)
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    page = pool.block_table[1, 2].item()
    assert (cache.k[page, :, :2] == 9).all() and torch.equal(cache.k[:2], k[:2])


def test_a_refused_fork_is_not_a_refused_reserve():
    from quantized_gemm_error_gb300 import spear
    pool, cache = _full_pool()
    spear.spear_kv_free(pool, _i(2))
    spear.spear_kv_reserve(pool, _i(1), _i(2))
    spear.spear_kv_fork(pool, cache, _i(0), _i(1))             # the child is in use
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 1
    spear.spear_kv_append(cache, _rows(2, 9), _rows(2, 9), pool.block_table, pool.seq_lens, _i(0, 2), seq_ids=_i(1), pool=pool)
    spear.spear_kv_fork(pool, cache, _i(1), _i(3))             # and one that is not
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    assert pool.seq_lens.tolist() == [8, 10, 0, 10] and pool.refs.tolist() == [3, 3, 1, 1]
    for row in (1, 3):
        assert (cache.k[pool.block_table[row, 2].item(), :, :2] == 9).all()


def test_a_server_that_runs_out_of_pages():
    from quantized_gemm_error_gb300 import spear
    from quantized_gemm_error_gb300.serve import AttentionBlock, PagedServer, PoolFull
    from test_gpu_serve import _layer
    block = lambda s: AttentionBlock(_layer(512, 256, s), _layer(512, 128, s + 1), _layer(512, 128, s + 2), _layer(256, 512, s + 3), 64)
    s = PagedServer([block(0), block(10)], 5, 16, 6, 8, "cuda")
    g = torch.Generator("cuda").manual_seed(1)
    x = lambda n: torch.randn(n, 512, generator=g, device="cuda").to(BF16)
    s.step(x(32), [0], [32])                                   # two whole pages
    s.fork([0], [1])
    s.step(x(46), [2], [46])                                   # the other three, the last one with room for two
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0 and s.count.free_pages == 0
    before = [t.clone() for c in s.caches for t in (c.k, c.v)] + [s.pool.snapshot()]

    def same():
        torch.cuda.synchronize()
        assert spear.spear_get_device_status() == 0            # nothing was launched
        assert all(torch.equal(a, b) for a, b in zip(before, [t for c in s.caches for t in (c.k, c.v)] + [s.pool.state]))

    for rows, counts in (([0], [1]), ([1, 2], [1, 1]), ([2], [3])):
        with pytest.raises(PoolFull):
            s.step(x(sum(counts)), rows, counts)
        same()
    with pytest.raises(PoolFull):
        s.fork([2], [3])
    for call in (lambda: s.step(x(2), [2, 2], [1, 1]), lambda: s.step(x(1), [6], [1]), lambda: s.step(x(200), [3], [200]),
                 lambda: s.step(x(1), [0, 2], [2, -1]), lambda: s.fork([0], [1]), lambda: s.finish([-1])):
        with pytest.raises(ValueError):
            call()
    same()
    s.step(x(2), [2], [2])                                     # what fits goes on
    s.finish([2])
    s.step(x(5), [0, 1], [1, 4])
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    assert s.pool.seq_lens.tolist() == [33, 36, 0, 0, 0, 0] == s.count.lens
    assert int((s.pool.refs == 0).sum()) == s.count.free_pages == 1
