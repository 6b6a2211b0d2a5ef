"""spear_kv_free with rows, lengths and counts that are wrong: reported, and nothing is lost."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _i(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _status():
    from quantized_gemm_error_gb300 import spear
    torch.cuda.synchronize()
    return spear.spear_get_device_status()


@pytest.mark.parametrize("length", [-1, 17, 1000, 2 ** 31 - 1])
def test_a_row_of_impossible_length_keeps_its_pages(length):
    from quantized_gemm_error_gb300 import spear
    pool = spear.PagePool(8, 4, 4, 4, "cuda")                # a row holds 16 tokens
    spear.spear_kv_reserve(pool, _i(0, 1, 2), _i(8, 4, 3))
    assert _status() == 0
    pool.seq_lens[0] = length
    before = pool.snapshot()
    spear.spear_kv_free(pool, _i(0, 0))
    assert _status() == 1 and torch.equal(pool.state, before)
    spear.spear_kv_free(pool, _i(1, 0))                      # the other one goes
    assert _status() == 1
    assert pool.seq_lens.tolist() == [length, 0, 3, 0] and pool.refs.tolist() == [1, 1, 0, 1, 0, 0, 0, 0]
    pool.seq_lens[0] = 8                                     # and with its length so does this
    spear.spear_kv_free(pool, _i(0))
    assert _status() == 0
    assert pool.seq_lens.tolist() == [0, 0, 3, 0] and pool.refs.tolist() == [0, 0, 0, 1, 0, 0, 0, 0]


def test_a_count_does_not_go_below_zero():
    from quantized_gemm_error_gb300 import spear
    pool = spear.PagePool(8, 4, 4, 4, "cuda")
    spear.spear_kv_reserve(pool, _i(0, 1), _i(12, 4))
    assert _status() == 0
    pool.refs[1] = 0                                         # a page that row 0 names and nobody holds
    pool.block_table[0, 2] = 99
    spear.spear_kv_free(pool, _i(0))
    assert _status() == 1
    assert pool.refs.tolist() == [0, 0, 1, 1, 0, 0, 0, 0] and pool.seq_lens.tolist() == [0, 4, 0, 0]
    pool.refs[2] = 0
    spear.spear_kv_reserve(pool, _i(2), _i(28 - 4 - 8))      # the free ones can be had, that page among them
    assert _status() == 0
    assert pool.refs.tolist() == [1, 1, 1, 1, 1, 0, 0, 0] and pool.block_table[2].tolist() == [0, 1, 2, 4]
    # rows that share pages, freed in one call
    pool = spear.PagePool(64, 1, 40, 8, "cuda")
    cache = spear.new_kv_cache(64, 1, 1, 64, "cuda")
    spear.spear_kv_reserve(pool, _i(0), _i(8))
    spear.spear_kv_fork(pool, cache, _i(*[0] * 39), _i(*range(1, 40)))
    assert _status() == 0 and pool.refs[:8].tolist() == [40] * 8
    spear.spear_kv_free(pool, _i(*range(40), *range(40)))
    assert _status() == 0 and int(pool.refs.abs().sum()) == 0
