"""The server's count of lengths and free pages against the Python model of the pool (CPU only)."""
import random

import pytest

from quantized_gemm_error_gb300.serve import PageCount, PoolFull
from test_gpu_kv_pages import Model


@pytest.mark.parametrize("P,page,rows,cols", [(12, 4, 6, 5), (40, 1, 9, 12), (200, 16, 20, 30), (7, 100, 4, 3)])
@pytest.mark.parametrize("seed", range(6))
def test_random_calls(P, page, rows, cols, seed):
    rng = random.Random(seed)
    model, count = Model(P, page, rows, cols), PageCount(P, page, rows, cols)
    refused = full = 0
    for _ in range(300):
        op = rng.choice(["reserve", "reserve", "reserve", "fork", "free", "compact"])
        if op == "reserve":
            r = [rng.randrange(rows) for _ in range(rng.randint(1, 4))]
            t = [rng.randint(0, 2 * page + 3) for _ in r]
            ok, call = model.reserve(r, t), lambda: count.reserve(r, t)
        elif op == "fork":
            c = [rng.randrange(rows) for _ in range(rng.randint(1, 3))]
            p = [rng.randrange(rows) for _ in c]
            ok, call = model.fork(p, c) is not None, lambda: count.fork(p, c)
        elif op == "free":
            r = [rng.randrange(rows) for _ in range(rng.randint(1, 3))]
            model.free(r)
            ok, call = True, lambda: count.free(r)
        else:
            model.compact()
            ok, call = True, lambda: None
        if ok:
            call()
        else:
            with pytest.raises((ValueError, PoolFull)) as e:
                call()
            refused += 1
            full += e.type is PoolFull
        assert count.lens == model.lens
        assert count.free_pages == len(model.free_list())
    assert refused and refused > full


def test_refusals_change_nothing():
    c = PageCount(4, 4, 4, 3)
    c.reserve([0, 1], [8, 3])
    state = lambda: (list(c.lens), [[list(r) for r in row] for row in c.runs], c.free_pages)
    before = state()
    with pytest.raises(PoolFull):
        c.reserve([0, 1], [1, 2])
    for rows, counts in (([0, 0], [1, 1]), ([4], [1]), ([-1], [1]), ([2], [-1]), ([2], [13]), ([2, 3], [1])):
        with pytest.raises(ValueError):
            c.reserve(rows, counts)
    for p, k in (([0], [1]), ([0, 0], [2, 2]), ([0, 2], [2, 3]), ([9], [2]), ([0], [2, 3])):
        with pytest.raises(ValueError):
            c.fork(p, k)
    with pytest.raises(PoolFull):
        c.fork([1, 1], [2, 3])
    with pytest.raises(ValueError):
        c.free([0, 4])
    assert state() == before


@pytest.mark.parametrize("seed", range(6))
def test_recount_takes_over_a_pools_state(seed):
    """A count made anew from lengths and table goes on like the one that was there all along."""
    rng = random.Random(seed)
    P, page, rows, cols = 60, 4, 8, 12
    model, count = Model(P, page, rows, cols), PageCount(P, page, rows, cols)
    for step in range(200):
        if step % 5 == 4:
            count = PageCount(P, page, rows, cols)
            count.recount(model.lens, [r + [-1] * (cols - len(r)) for r in model.table])
            assert count.lens == model.lens and count.free_pages == len(model.free_list())
        op = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        r = rng.sample(range(rows), 2)
        if op == "reserve":
            t = [rng.randint(0, 9) for _ in r]
            ok, call = model.reserve(r, t), lambda: count.reserve(r, t)
        elif op == "fork":
            ok, call = model.fork(r[:1], r[1:]) is not None, lambda: count.fork(r[:1], r[1:])
        elif op == "free":
            model.free(r[:1])
            ok, call = True, lambda: count.free(r[:1])
        else:
            model.compact()
            continue
        if ok:
            call()
        else:
            with pytest.raises((ValueError, PoolFull)):
                call()
        assert count.lens == model.lens and count.free_pages == len(model.free_list())
