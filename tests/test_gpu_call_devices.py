"""Attention and cache calls refuse tensors that are not on the device of the cache or pool.  Stand-ins that say they are
on cuda:1 take the place of each argument in turn; nothing is launched with them."""
import pytest
import torch

from attn_testutil import Case

pytestmark = pytest.mark.gpu


class Elsewhere:
    """A tensor that says it is on cuda:1."""

    def __init__(self, t):
        self._t = t

    device, is_cuda = torch.device("cuda", 1), True

    def get_device(self):
        return 1

    def __getattr__(self, name):
        return getattr(self._t, name)


def _calls():
    from quantized_gemm_error_gb300 import spear
    c = Case([40, 90], [3, 4], Hq=4, Hkv=2, D=64)
    cache = c.cache()
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pool = spear.PagePool(c.num_pages, 16, 4, 8, "cuda")
    ws = spear.new_workspace(spear.spear_attn_decode_workspace_bytes(cache, 2, 4) +
                             spear.spear_attn_prefill_workspace_bytes(cache, 2, 7, 4), "cuda")
    common = dict(cache=cache, block_table=c.table, seq_lens=c.seq_lens, seq_ids=i(0, 1))
    attn = lambda n: dict(q=c.q_dev[:n], out=torch.empty_like(c.q_dev[:n]), lse=torch.empty(n, 4, device="cuda"),
                          workspace=ws)
    new = c.q_dev[:, :2].contiguous()
    return {
        spear.spear_attn_decode: {**common, **attn(2)},
        spear.spear_attn_prefill: {**common, **attn(7), "starts": c.starts},
        spear.spear_kv_append: {**common, "k_new": new, "v_new": new.clone(), "starts": c.starts},
        spear.spear_kv_reserve: dict(pool=pool, rows=i(0), tokens=i(3)),
        spear.spear_kv_fork: dict(pool=pool, caches=cache, parents=i(0), children=i(1)),
        spear.spear_kv_free: dict(pool=pool, rows=i(1)),
        spear.spear_kv_compact: dict(pool=pool, caches=[cache]),
        spear.spear_kv_copy_pages: dict(caches=[cache], moves=i(0, 0, 1, 2)),
    }


def test_every_argument_has_to_be_on_the_device():
    from quantized_gemm_error_gb300 import spear
    calls = _calls()
    for f, kw in calls.items():
        f(**kw)                                              # all right as they are
    torch.cuda.synchronize()
    assert spear.spear_get_device_status() == 0
    tried = 0
    for f, kw in calls.items():
        for name, value in kw.items():
            if isinstance(value, torch.Tensor):
                with pytest.raises(ValueError, match="cuda"):
                    f(**{**kw, name: Elsewhere(value)})
                tried += 1
        for name in ("cache", "caches", "pool"):
            obj = kw.get(name)
            obj = obj[0] if isinstance(obj, list) else obj
            if obj is not None:
                obj.index = 1
                try:
                    with pytest.raises(ValueError, match="cuda"):
                        f(**kw)
                finally:
                    obj.index = 0
    assert tried >= 24
    with pytest.raises(ValueError, match="cuda"):
        kw = calls[spear.spear_kv_append]
        pool = spear.PagePool(4, 4, 4, 4, "cuda")
        pool.index = 1
        spear.spear_kv_append(**kw, pool=pool)


def test_the_current_device_and_the_stream_have_to_be_the_caches(monkeypatch):
    calls = _calls()
    torch.cuda.synchronize()

    class Stream:
        device_index, cuda_stream = 1, 0

    for f, kw in calls.items():
        with pytest.raises(ValueError, match="stream"):
            f(**kw, stream=Stream())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for f, kw in calls.items():
        with pytest.raises(ValueError, match="current device"):
            f(**kw)
