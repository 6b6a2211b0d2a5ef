"""spear_get_device_status: every kind of kernel's word is read and cleared, once, whichever thread asks."""
import threading

import pytest
import torch

from attn_testutil import Case

pytestmark = pytest.mark.gpu


def _errors():
    """Calls whose kernels report SPEAR_ERR_INVALID_ARG, by the file that holds the word."""
    from quantized_gemm_error_gb300 import spear
    W = torch.randn(512, 1024, device="cuda") / 32
    q, s, z = spear.spear_pack_w4(W, 128, False)
    layer = spear.W4Layer(512, 1024, 128, False, q, s, z)
    bad_w = W.clone()
    bad_w[3, 5] = float("nan")
    x = torch.ones(300, 1024, dtype=torch.bfloat16, device="cuda")
    x[0, 7] = float("inf")
    c = Case([40, 90], [3, 4], Hq=4, Hkv=2, D=64)
    cache, lens = c.cache(), c.seq_lens.clone()
    lens[0] = -1
    pool = spear.PagePool(4, 4, 4, 4, "cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    row, n = i(2), i(100)
    torch.cuda.synchronize()
    return {
        "pack": lambda: spear.spear_pack_w4(bad_w, 128, False),
        "decode of 3": lambda: spear.spear_linear_decode(layer, x[:3]),
        "decode of 40": lambda: spear.spear_linear_decode(layer, x[:40]),
        "prefill": lambda: spear.spear_linear_prefill(layer, x),
        "pool": lambda: spear.spear_kv_reserve(pool, row, n),
        "attn_decode": lambda: spear.spear_attn_decode(c.q_dev[:2], cache, c.table, lens),
        "attn_prefill": lambda: spear.spear_attn_prefill(c.q_dev, cache, c.table, lens, c.starts),
    }


def test_each_word_is_read_once():
    from quantized_gemm_error_gb300 import spear
    errors = _errors()
    assert spear.spear_get_device_status() == 0
    for name, call in errors.items():
        call()
        assert spear.spear_get_device_status() == 1, name
        assert spear.spear_get_device_status() == 0, name
    for call in errors.values():                             # all at once: one read takes them all
        call()
    assert spear.spear_get_device_status() == 1
    assert spear.spear_get_device_status() == 0


def test_on_a_side_stream_and_from_several_threads():
    from quantized_gemm_error_gb300 import spear
    call = _errors()["pool"]
    for round_ in range(20):
        call()
        torch.cuda.synchronize()
        seen, streams = [], [torch.cuda.Stream() for _ in range(4)]

        def ask(st):
            for _ in range(5):
                seen.append(spear.spear_get_device_status(st))

        threads = [threading.Thread(target=ask, args=(st,)) for st in streams]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert sorted(seen) == [0] * 19 + [1], round_
