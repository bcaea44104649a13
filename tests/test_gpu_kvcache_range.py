"""The paged key-value cache at the ends of its number ranges, through the C ABI.

Decoded outputs are compared with the fp64 golden under the bound of test_gpu_kvcache, whose terms count each
rounding, plus 2^-16 of sum p|v|: a weight's exponent here is up to 2^8 in magnitude (score and scale), so its
fp32 sums round by up to 2^-17 each, twice.
"""

import numpy as np
import pytest
import torch

import mixture_transformers_token_gb300 as mot
from mixture_transformers_token_gb300 import workloads as W
from oracle import mot_oracle as O

from _util import f64, need_gpu
from test_gpu_kvcache import DEV, E4M3, Batch, _bound, _empty_cache, _ws

pytestmark = pytest.mark.gpu

BF16_MAX = float(torch.finfo(torch.bfloat16).max)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _rewrite(b):
    """Writes the rows b.x into the batch's cache again."""
    tab = b.table.cpu().numpy()
    for r, x in enumerate(b.x):
        if len(x):
            j = np.arange(len(x))
            slots = (tab[r, j // b.page].astype(np.int64) * b.page + j % b.page).astype(np.int32)
            mot.mot_kv_cache_write(x.to(DEV), torch.from_numpy(slots).to(DEV), b.k, b.v, b.Hq, _ws(), scales=b.scales)


def _check(b, what):
    out = b.run()
    g = b.golden()
    got = f64(out).reshape(g["out_pre"].shape)
    d = np.abs(got - g["out_pre"])
    bound = _bound(g, b.lens, b.D, b.kv) + 2.0 ** -16 * g["p_abs_v"]
    assert np.isfinite(got).all(), f"{what}: {np.argwhere(~np.isfinite(got))[:5]}"
    assert np.all(d <= bound), f"{what}: {np.argwhere(d > bound)[:5]} worst {np.max(d / bound):.3g} of the bound"
    return out


# keys of a row, the loud key's place: one tile, another warp of the item, another range of the row
PLACES = [(2, 0), (2, 1), (64, 40), (300, 0), (1500, 5), (1500, 1499), (20000, 9000)]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,at", PLACES)
@pytest.mark.parametrize("top", [60, 90, 104, 119])
def test_one_loud_value_among_quiet_ones_keeps_the_others_in_the_sum(kv, n, at, top):
    # equal scores: the output is the mean of the values, whatever their scales; the quiet values are zeros (the
    # smallest scale there is) or of unit size
    D = 128 if top % 2 else 64
    Hq, Hkv = (20, 2) if n == 300 else (2, 1)
    for zeros in (True, False):
        b = Batch([n, 3], Hq, Hkv, D, kv, 16, seed=n + top, q_gain=0.0)
        x = b.x[0].float()
        v = x[:, (Hq + Hkv) * D:]
        if zeros:
            v[:] = 0.0
        v[at] = 1.5 * 2.0 ** top * torch.where(torch.arange(Hkv * D) % 3 == 0, -1.0, 1.0)
        b.x[0] = x.to(torch.bfloat16)
        _rewrite(b)
        _check(b, f"2^{top} at {at} of {n}, zeros {zeros}")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,at", PLACES)
@pytest.mark.parametrize("lead", [10.0, 60.0, 95.0])
def test_a_loud_value_whose_key_has_next_to_no_weight(kv, n, at, lead):
    # the other keys lead by `lead` powers of two, and the loud value's share still outweighs theirs
    Hq, Hkv, D = 2, 1, 128
    b = Batch([n], Hq, Hkv, D, kv, 16, seed=n + int(lead))
    x = b.x[0].float()
    q = torch.zeros(D)
    q[:64] = 1.0
    b.q[:, : Hq * D] = torch.cat([q, q]).to(torch.bfloat16).to(DEV)
    # scores: 64 k / sqrt(128) nats
    x[:, Hq * D: (Hq + Hkv) * D] = 0.0
    x[at, Hq * D: Hq * D + 64] = -lead * np.log(2.0) * np.sqrt(128.0) / 64
    x[:, (Hq + Hkv) * D:] *= 2.0 ** -20
    x[:, (Hq + Hkv) * D:][at] = 1.25 * 2.0 ** 118
    b.x[0] = x.to(torch.bfloat16)
    _rewrite(b)
    _check(b, f"lead {lead} at {at} of {n}")


@pytest.mark.parametrize("n,at", PLACES)
def test_scales_at_both_ends_of_their_range(n, at):
    # scales of 2^-64 beside one of 2^126, code 1, equal scores
    Hq, Hkv, D, page = 3, 1, 64, 16
    b = Batch([n], Hq, Hkv, D, "e4m3", page, seed=5, q_gain=0.0)
    b.v.copy_(torch.ones(b.v.shape, device=DEV).to(E4M3))
    b.scales[..., 1] = 2.0 ** -64
    b.scales[int(b.table[0, at // page]), 0, at % page, 1] = 2.0 ** 126
    want = 2.0 ** 126 / n   # + (n - 1) 2^-64 / n
    got = f64(b.run())
    assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) * want), got[0, 0] / want


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 5, 64, 700, 3000, 20000])
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_the_types_largest_size_do_not_overflow(n, D, kv):
    # an output is a mean of values: finite wherever they are. e4m3 holds 1.75 2^127 exactly, bf16 its largest value
    Hq, Hkv = 3, 1
    top = BF16_MAX if kv == "bf16" else 1.75 * 2.0 ** 127
    for gain, rising in ((0.0, False), (1.0, False), (1.0, True)):
        b = Batch([n, 2], Hq, Hkv, D, kv, 16, seed=n + D, q_gain=gain)
        for r, x in enumerate(b.x):
            x = x.float()
            if rising:  # scores that rise with the keys, so that a reference lags behind and moves
                q = b.q[r, :D].float().cpu()
                x[:, Hq * D: (Hq + Hkv) * D] = q[None, :] * (torch.arange(len(x))[:, None] / len(x) * 4.0)
            v = x[:, (Hq + Hkv) * D:]
            v[:] = torch.where(torch.arange(D) % 3 == 0, -top, top)
            b.x[r] = x.to(torch.bfloat16)
        _rewrite(b)
        _check(b, f"gain {gain}, rising {rising}")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("up,down", [(119, -58), (127, -60), (-126, 100)])
def test_queries_and_keys_of_opposite_sizes(up, down, kv):
    # every score is exact in fp32 and far below its end, although a factor of it may be near an end of the range.
    # Large ones: the even keys share the row, the odd ones have nothing; tiny ones: every key has the same weight
    Hq, Hkv, D = 4, 2, 128
    b = Batch([70, 1200], Hq, Hkv, D, kv, 16, seed=200 + up)
    sign = torch.where(torch.arange(D) % 5 == 0, -1.0, 1.0)
    b.q[:, : Hq * D] = (sign.repeat(Hq) * 2.0 ** up).to(torch.bfloat16).to(DEV)
    for r, x in enumerate(b.x):
        x = x.float()
        each = torch.where(torch.arange(len(x))[:, None] % 2 == 0, 1.0, 0.75) * 2.0 ** down
        x[:, Hq * D: (Hq + Hkv) * D] = sign.repeat(Hkv)[None, :] * each
        b.x[r] = x.to(torch.bfloat16)
    _rewrite(b)
    got = f64(b.run()).reshape(2, Hq, D)
    for r, x in enumerate(b.x):
        v = f64(x)[:, (Hq + Hkv) * D:].reshape(-1, Hkv, D)
        if kv == "e4m3":
            y, s = O.kv_quantise(v)
            v = y * s[..., None]
        if up > 0:
            v = v[::2]
        want, mean_abs = v.mean(0), np.abs(v).mean(0)
        # the output's rounding; a weight's, and a handful of fp32 factors; the sums
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -16 + 4 * len(v) * 2.0 ** -24) * mean_abs
        # e4m3: the exponent of a weight is the score, here about 2^65 (or 2^71) with a spacing of 2^42, plus log2 of
        # its V scale, at most 2^8: that sum rounds to the score, so that the keys' weights p differ by up to the ratio
        # of their scales, which the bound's 2^-22 |s| = 2^43 covers. Both sums take the same p >= 0, so the output is
        # some mean of the even keys' values: within their hull, a half's and a bf16's rounding aside
        any_mean = kv == "e4m3" and up > 0
        slack = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16 + 4 * len(v) * 2.0 ** -24) * np.abs(v).max(0)
        for h in range(Hq):
            g, o = h // 2, got[r, h]
            if any_mean:
                assert np.all(o >= v.min(0)[g] - slack[g]) and np.all(o <= v.max(0)[g] + slack[g]), (r, h)
            else:
                assert np.all(np.abs(o - want[g]) <= bound[g]), (r, h)


def test_read_back_rounds_once_whatever_the_scale():
    # code * scale has up to 28 bits: scales for which rounding it to fp32 and then to bf16 would differ from rounding
    # it to bf16 at once, every code with each
    Hkv, D, page = 1, 128, 16
    r = W.rng_for(9, 609)
    s = (r.integers(1 << 23, 1 << 24, 1 << 20).astype(np.float64) * 2.0 ** -23)
    odd = []
    for m in (9.0, 11.0, 13.0, 15.0):
        twice = O.bf16((s * m).astype(np.float32).astype(np.float64))
        odd.append(s[twice != O.bf16(s * m)])
    odd = np.concatenate(odd)[:32]
    assert len(odd) >= 8
    scales = np.concatenate([odd * np.exp2(r.integers(-60, 100, len(odd))), np.exp2(r.uniform(-60, 100, 64 - len(odd)))])
    scales = scales.astype(np.float32)
    codes = np.arange(128, dtype=np.uint8)
    codes[127] = 0x7E
    codes = np.concatenate([codes, codes | 0x80])
    k, v, sc = _empty_cache(64 // page, Hkv, page, D, "e4m3")
    k.view(torch.uint8).copy_(torch.from_numpy(codes[:128]).to(DEV).expand(k.shape))
    v.view(torch.uint8).copy_(torch.from_numpy(codes[128:]).to(DEV).expand(v.shape))
    sc[..., 0] = torch.from_numpy(scales).to(DEV).reshape(sc.shape[:-1])
    sc[..., 1] = torch.from_numpy(scales[::-1].copy()).to(DEV).reshape(sc.shape[:-1])
    ws = _ws()
    y = torch.zeros((64, 3 * D), dtype=torch.bfloat16, device=DEV)
    mot.mot_kv_cache_read(k, v, torch.arange(64, dtype=torch.int32, device=DEV), y, 1, ws, scales=sc)
    assert mot.mot_device_status(ws) == 0
    vals = k.to(torch.float32).cpu().numpy()[0, 0, 0].astype(np.float64)
    got = f64(y)
    np.testing.assert_array_equal(got[:, D: 2 * D], O.bf16(vals[None, :] * scales.astype(np.float64)[:, None]))
    np.testing.assert_array_equal(got[:, 2 * D:], O.bf16(-vals[None, :] * scales.astype(np.float64)[::-1, None]))


def test_a_refused_call_leaves_a_capture_usable():
    # the stream's device is asked for while it is being captured, and a pointer of no device is refused there
    Hq, Hkv, D, page, T = 2, 1, 64, 16, 20
    x = W.bf16_normal(W.rng_for(3, 611), (T, (Hq + 2 * Hkv) * D)).to(DEV)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    k, v, _ = _empty_cache(2, Hkv, page, D, "bf16")
    ws, host = _ws(), np.zeros(64, np.uint8)
    at = (host.ctypes.data + 15) // 16 * 16
    side, graph, lib = torch.cuda.Stream(), torch.cuda.CUDAGraph(), mot.load_library()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        mot.mot_kv_cache_write(x, slots, k, v, Hq, ws)
        # qkv in host memory
        assert lib.mot_kv_cache_write(at, 1, Hq, Hkv, D, slots.data_ptr(), mot.KV_BF16, 2, page, k.data_ptr(),
                                      v.data_ptr(), None, ws.data_ptr(), 64, side.cuda_stream) == 4
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert mot.mot_device_status(ws) == 0
    got = k.transpose(1, 2).reshape(-1, D)[:T]
    assert torch.equal(got, x[:, Hq * D: (Hq + 1) * D])
