"""The paged key-value cache's binding: what is no tensor, or one of the wrong rank, is refused by name."""

import pytest
import torch

import mixture_transformers_token_gb300 as mot

from _util import need_gpu

DEV = "cuda"


@pytest.mark.parametrize("what", [None, 3, "k", [1.0]])
def test_a_cache_that_is_no_tensor(what):
    x = torch.zeros(1, 64)
    for call in (lambda: mot.mot_kv_cache_write(x, x, what, x, 1, x), lambda: mot.mot_kv_cache_read(what, x, x, x, 1, x),
                 lambda: mot.mot_paged_decode_attention(x, x, x, what, x, 1, x)):
        with pytest.raises(TypeError, match="k_cache"):
            call()


def test_a_cache_on_the_host():
    k = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_cache must be a CUDA tensor"):
        mot.mot_kv_cache_write(k, k, k, k, 1, k)


@pytest.mark.gpu
def test_each_argument_by_name():
    need_gpu()
    Hq, D, page = 2, 64, 16
    good = dict(qkv=torch.zeros((3, 4 * D), dtype=torch.bfloat16, device=DEV),
                slots=torch.arange(3, dtype=torch.int32, device=DEV),
                k_cache=torch.zeros((2, 1, page, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                v_cache=torch.zeros((2, 1, page, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                scales=torch.ones((2, 1, page, 2), device=DEV),
                table=torch.zeros((3, 2), dtype=torch.int32, device=DEV),
                lens=torch.ones(3, dtype=torch.int32, device=DEV),
                ws=torch.zeros(1 << 16, dtype=torch.uint8, device=DEV))

    def calls(**kw):
        a = {**good, **kw}
        rows = dict(qkv=a["qkv"], slots=a["slots"], k_cache=a["k_cache"], v_cache=a["v_cache"], Hq=Hq, ws=a["ws"],
                    scales=a["scales"])
        dec = {**rows, "table": a["table"], "lens": a["lens"]}
        del dec["slots"]
        return ((mot.mot_kv_cache_write, rows), (mot.mot_kv_cache_read, rows), (mot.mot_paged_decode_attention, dec))

    for f, kw in calls():
        f(**kw)
    assert mot.mot_device_status(good["ws"]) == 0
    for name in good:
        for bad, error in ((7, TypeError), ("x", TypeError), (good[name].double(), TypeError),
                           (good[name].cpu(), ValueError), (good[name].unsqueeze(0), ValueError)):
            for f, kw in calls(**{name: bad}):
                if name in kw:
                    with pytest.raises(error, match=name):
                        f(**kw)
