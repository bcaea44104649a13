"""The 8-bit AdamW states' codes byte by byte, above all in blocks whose scale is zero or a NaN, and the bf16 copies element by
element: a comparison of values takes a code of minus zero for one of zero."""

import numpy as np
import pytest
import torch

import mixture_transformers_token_gb300 as mot
from oracle import mot_oracle as O

from _util import bits, need_gpu
from test_gpu_adamw import Case, _hyper, _ws

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _codes(values, scale):
    """Bytes of the emulator's e4m3 values; of a block whose scale is zero or a NaN, zero."""
    c = torch.from_numpy(np.asarray(values, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    c[~np.repeat(scale > 0, 256)[:c.size]] = 0
    return c


def _check(c, want):
    for i, (p, m, v, s) in enumerate(want):
        got = c.p[i].cpu().numpy()
        fine = ~np.isnan(p)
        assert np.array_equal(np.isnan(got), ~fine) and np.array_equal(got[fine].view(np.int32), p[fine].view(np.int32))
        assert np.array_equal(bits(c.p16[i])[fine], bits(torch.from_numpy(p).to(torch.bfloat16))[fine])
        assert bool(torch.isnan(c.p16[i].cpu()[torch.from_numpy(~fine)]).all())
        got = c.scales[i].cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(s)) and np.array_equal(got[~np.isnan(s)], s[~np.isnan(s)])
        for state, w, k in ((c.m[i], m, 0), (c.v[i], v, 1)):
            a, b = state.view(torch.uint8).cpu().numpy(), _codes(w, s[:, k])
            bad = np.flatnonzero(a != b)
            assert bad.size == 0, (i, "mv"[k], bad.size, bad[:4] // 256, a[bad[:4]], b[bad[:4]], s[bad[:4] // 256, k])


def _steps(c, steps, seed=3):
    for t in steps:
        want = c.want(t, 1.0, seed)
        mot.mot_adamw_step(c.plan, _hyper(t), _ws(), seed=seed)
        _check(c, want)


@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [255, 256, 257], [100003, 5]], ids=lambda s: f"{len(s)}x{max(s)}")
def test_codes_of_ordinary_steps(sizes, grad):
    _steps(Case(sizes, "e4m3", grad, seed=len(sizes)), (1, 2, 1000003))


def test_a_block_whose_squares_all_overflow():
    # the first moment is even and finite, so that it alone would take the rounding without subnormals
    c = Case([256 * 6 + 100], "e4m3", seed=7)
    for k, x in enumerate((1e25, -1e25, 3e20, 2e38)):
        c.g[0][256 * k:256 * (k + 1)] = x
    c.g[0][256 * 6:] = 1e25  # and a block that is not whole
    want = c.want(1, 1.0, 3)[0]
    assert np.isnan(want[3][[0, 1, 2, 3, 6], 1]).all() and np.isfinite(want[3][[0, 1, 2, 3, 6], 0]).all()
    _steps(c, (1, 2))


def test_the_step_after_one_square_overflowed():
    # its block's scale is a NaN, so that every second moment of the block becomes one
    c = Case([256 * 3], "e4m3", seed=8)
    c.g[0][300] = 1e25
    _steps(c, (1,))
    c.g[0][256:512] = 1e-3 * torch.sign(c.g[0][256:512])  # beside a first moment without small values
    c.m[0].view(torch.uint8)[256:512] = 0
    _steps(c, (2, 3))
    got = c.scales[0].cpu().numpy()
    assert np.isnan(got[1, 1]) and np.isfinite(got[[0, 2]]).all()
    assert bool(torch.isnan(c.p[0][256:512]).all()) and bool(torch.isfinite(c.p[0][:256]).all())


def test_first_moments_that_are_nan_beside_second_ones_that_are_not():
    c = Case([512], "e4m3", seed=9)
    c.g[0].fill_(1e-3)
    c.scales[0][1, 0] = float("nan")
    _steps(c, (1, 2))
    assert np.isnan(c.scales[0].cpu().numpy()[1, 0]) and np.isfinite(c.scales[0].cpu().numpy()[1, 1])


def test_blocks_below_the_least_scale():
    # magnitudes under 2^-100 of either sign: scale and codes are zero
    c = Case([256 * 3 + 9], "e4m3", seed=10)
    c.g[0][:256] = -(2.0 ** -105)
    c.g[0][256:512] *= 2.0 ** -110
    c.g[0][768:] *= 2.0 ** -120
    _steps(c, (1, 2))
    assert not c.scales[0].cpu().numpy()[[0, 1, 3]].any()
    assert not c.m[0].view(torch.uint8)[:512].any() and not c.m[0].view(torch.uint8)[768:].any()
