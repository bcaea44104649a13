"""The softmax scale that the single-token attention accepts: its product with log2 e is finite in fp32."""

import numpy as np

from test_kvcache_host import MOT_ERR_ARG, _cache_calls, lib  # noqa: F401 (lib: the fixture)


def test_a_scale_whose_product_with_log2_e_overflows_is_refused(lib):  # noqa: F811
    f = _cache_calls(lib)[2]
    log2e = np.float32(1.4426950408889634)
    for scale in (np.float32(2.5e38), np.float32(2.9e38), np.finfo(np.float32).max / log2e * np.float32(1.0001)):
        with np.errstate(over="ignore"):
            assert np.isinf(np.float32(scale) * log2e)
        assert f(scale=float(scale)) == MOT_ERR_ARG, scale
    for scale in (1e-45, 1.0, np.finfo(np.float32).max / log2e * np.float32(0.9999)):
        assert np.isfinite(np.float32(scale) * log2e)
        assert f(scale=float(scale)) not in (0, MOT_ERR_ARG), scale   # what is left to fail is the device
