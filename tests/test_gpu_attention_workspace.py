"""The binding's own workspaces of the attention calls: their size does not depend on a call's, and what a cache keeps
does not grow with the calls made on it."""
import pytest
import torch

from attn_testutil import Case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_sizes_do_not_depend_on_the_call(D):
    from quantized_gemm_error_gb300 import spear
    cache = spear.new_kv_cache(4, 16, 2, D, "cuda")
    assert len({spear.spear_attn_decode_workspace_bytes(cache, b, h) for b in (0, 1, 33, 5000) for h in (2, 8, 256)}) == 1
    assert len({spear.spear_attn_prefill_workspace_bytes(cache, b, t, h) for b in (1, 700) for t in (1, 9, 8192, 10 ** 6)
                for h in (2, 8, 256)}) == 1


def test_what_a_cache_keeps_does_not_grow():
    from quantized_gemm_error_gb300 import spear
    spear.reset_default_workspaces()
    cases = [Case([n, 40], [n, 3], Hq=h, Hkv=2, D=128, seed=n) for n, h in ((3, 2), (50, 8), (200, 6), (7, 16))]
    cache = None
    for c in cases:
        cache = c.cache()
        for n in range(1, 4):
            out = spear.spear_attn_prefill(c.q_dev, cache, c.table, c.seq_lens, c.starts)
            one = spear.spear_attn_decode(c.q_dev[:n], cache, c.table[:1].expand(n, -1).contiguous(),
                                          c.seq_lens[:1].expand(n).contiguous())
            assert one.shape[0] == n
        torch.cuda.synchronize()
        check(out, None, c.reference(), "prefill")
    kept = lambda: sum(len(v) for v in vars(cache).values() if isinstance(v, (dict, list, set, tuple)))
    before = kept()
    for t in range(1, 60):
        starts = torch.tensor([0, t], dtype=torch.int32, device="cuda")
        q = torch.zeros(t, 2 + 2 * (t % 5), 128, dtype=cache.dtype, device="cuda")
        spear.spear_attn_prefill(q, cache, c.table[:1], c.seq_lens[:1], starts)
        if t > 1:
            spear.spear_attn_decode(q[:2], cache, c.table, c.seq_lens)
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    assert kept() == before
