"""Decode over every key of a row once, and what only a loud row or a quantised prefix reaches, through the C ABI."""

import numpy as np
import pytest
import torch

import mixture_transformers_token_gb300 as mot
from oracle import mot_oracle as O

from _util import assert_bitwise, f64, need_gpu
from test_gpu_kvcache import DEV, Batch, _empty_cache, _kv, _qkv, _slots, _ws
from test_gpu_kvcache_range import PLACES, _check, _rewrite

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,D,page", [(33, 64, 16), (700, 128, 16), (4100, 64, 48), (20011, 128, 32), (40000, 128, 64)])
def test_every_key_counts_once(n, D, page, kv):
    # equal scores and values of 0 and 1: dim d of pass p is 1 in the keys of one block, at most 40, so the output is
    # that block's share of the row, to a bf16's rounding. A key that is lost or counted twice changes it by 2.5 %,
    # and one that is missing from the sum of the weights alone changes every dim
    Hq, Hkv, block = 3, 1, 40
    b = Batch([n], Hq, Hkv, D, kv, page, seed=n, q_gain=0.0)
    keys = np.arange(n)
    at = torch.from_numpy(b.table.cpu().numpy()[0, keys // page].astype(np.int64) * page + keys % page).to(DEV)
    if kv == "e4m3":
        b.scales[..., 1] = 1.0
    blocks = -(-n // block)
    size = np.bincount(keys // block, minlength=blocks).astype(np.float64)
    err = 2.0 ** -8 + 2.0 ** -16
    assert (1.0 / size > 4 * err).all()
    for p0 in range(0, blocks, D):
        v = torch.zeros((n, D), device=DEV)
        mine = torch.arange(n, device=DEV) // block - p0
        on = (mine >= 0) & (mine < D)
        v[on, mine[on]] = 1.0
        b.v.zero_() if kv == "bf16" else b.v.view(torch.uint8).zero_()
        flat = b.v.reshape(-1, D) if kv == "bf16" else b.v.view(torch.uint8).reshape(-1, D)
        flat[at] = v.to(b.v.dtype) if kv == "bf16" else v.to(b.v.dtype).view(torch.uint8)
        want = np.zeros(D)
        want[: min(D, blocks - p0)] = size[p0: p0 + D] / n
        one = b.run()
        got = f64(one).reshape(Hq, D)
        assert np.all(np.abs(got - want) <= err * want), (p0, np.argwhere(np.abs(got - want) > err * want)[:5])
        # the other form of the join
        many = b.run([0] * 400)
        assert_bitwise(many, one.expand(400, -1).contiguous(), "many rows")


def _loud_batch(seed, n_pages=None):
    """Rows with a value of 2^60 to 2^110 in their first, a middle or their last key, among ordinary rows."""
    lens = [900, 1, 0, 77, 3000, 256, 13, 512]
    b = Batch(lens, 14, 2, 128, "e4m3", 16, seed=seed, n_pages=n_pages)
    for r, (at, top) in {0: (450, 60), 1: (0, 100), 4: (2999, 110), 6: (0, 80)}.items():
        x = b.x[r].float()
        x[at, (b.Hq + b.Hkv) * b.D:] *= 2.0 ** top
        b.x[r] = x.to(torch.bfloat16)
    _rewrite(b)
    return b


def test_loud_rows_bits_do_not_depend_on_the_batch():
    b = _loud_batch(211)
    want = _check(b, "loud rows")
    assert_bitwise(b.run(), want, "repeat")
    for rows in ([4], [0], [1], [3, 5], [7, 6, 5, 4, 3, 2, 1, 0], [4] * 9, [4, 0] * 200):
        assert_bitwise(b.run(rows), want[torch.tensor(rows, device=DEV)], f"rows {rows[:9]}")
    c = _loud_batch(211, n_pages=b.n_pages + 50)
    c.table = torch.cat([c.table, torch.full((8, 3000), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    assert_bitwise(c.run(), want, "another placement")
    ws, out = b.ws(), torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            mot.mot_paged_decode_attention(b.q, b.table, b.lens_t, b.k, b.v, b.Hq, ws, scales=b.scales, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert_bitwise(out, want, "replayed")
    assert mot.mot_device_status(ws) == 0


def test_loud_rows_with_a_bad_page_or_a_nan():
    b = _loud_batch(212)
    want = _check(b, "loud rows")
    others = [0, 1, 2, 3, 5, 6, 7]
    for entry in (-1, b.n_pages, 2 ** 31 - 1):
        t = b.table.clone()
        t[4, 187] = entry   # the loud key's own page
        t[4, 3] = entry
        ws = b.ws()
        out = mot.mot_paged_decode_attention(b.q, t, b.lens_t, b.k, b.v, b.Hq, ws, scales=b.scales)
        assert mot.mot_device_status(ws) == mot.DEV_BAD_PAGE
        assert torch.equal(out[others], want[others])
    # a NaN among the keys of one head of the loud row, then in one query
    x = b.x[4].clone()
    x[100, b.Hq * b.D + b.D + 3] = float("nan")
    clean, b.x[4] = b.x[4], x
    _rewrite(b)
    got, ref = f64(b.run()).reshape(8, 14, 128), f64(want).reshape(8, 14, 128)
    assert np.isnan(got[4, 7:]).all() and np.array_equal(got[4, :7], ref[4, :7]) and np.array_equal(got[others], ref[others])
    b.x[4] = clean
    _rewrite(b)
    b.q[4, 5 * 128 + 1] = float("nan")
    got = f64(b.run()).reshape(8, 14, 128)
    assert np.isnan(got[4, 5]).all() and np.array_equal(np.delete(got[4], 5, 0), np.delete(ref[4], 5, 0))


def test_joint_attention_over_a_prefix_read_from_a_quantised_cache():
    # the second chunk's joint attention over a prefix that comes back from an e4m3 cache gives the same bits as over
    # rows that hold the prefix's quantised values
    Hq, Hkv, D, n, pre, page = 4, 2, 128, 300, 211, 32
    x = _qkv(n, Hq, Hkv, D, 93).to(DEV)
    seqs = torch.tensor([[pre, 0, n - pre, n, 40]], dtype=torch.int32, device=DEV)
    ws = _ws()
    k, v, sc = _empty_cache(10, Hkv, page, D, "e4m3")
    slots = torch.from_numpy(_slots(pre, 320, 94)).to(DEV)
    mot.mot_kv_cache_write(x[:pre], slots, k, v, Hq, ws, scales=sc)
    y = torch.zeros_like(x)
    y[pre:] = x[pre:]
    mot.mot_kv_cache_read(k, v, slots, y[:pre], Hq, ws, scales=sc)
    got = mot.mot_joint_attention(y, seqs, Hq, Hkv, D, ws)
    z = x.clone()
    for i, a in enumerate(_kv(x[:pre], Hq, Hkv, D)):
        q, s = O.kv_quantise(a)
        at = (Hq + i * Hkv) * D
        z[:pre, at: at + Hkv * D] = torch.from_numpy((q * s[..., None]).reshape(pre, -1)).to(torch.bfloat16).to(DEV)
    want = mot.mot_joint_attention(z, seqs, Hq, Hkv, D, ws)
    assert mot.mot_device_status(ws) == 0
    assert_bitwise(got[pre:], want[pre:], "second chunk")


@pytest.mark.parametrize("n,at", PLACES)
@pytest.mark.parametrize("top", [24, 25])
def test_either_side_of_the_scale_from_which_sums_stand_apart(n, at, top):
    # one value with a V scale of 2^16 or 2^17 among zero vectors (2^-64) or values of 2^-50; its key is behind the
    # others' by up to 2^35, or leads
    Hq, Hkv, D = 2, 1, 64
    for lead in (0.0, 12.0, 35.0, -20.0):
        for quiet in (0.0, 2.0 ** -50):
            b = Batch([n, 2], Hq, Hkv, D, "e4m3", 16, seed=n + top)
            b.q[:, : Hq * D] = 1.0
            x = b.x[0].float()
            x[:, Hq * D:] = 0.0
            x[at, Hq * D: (Hq + Hkv) * D] = -lead * np.log(2.0) * np.sqrt(float(D)) / D
            x[:, (Hq + Hkv) * D:] = quiet
            x[at, (Hq + Hkv) * D:] = 1.5 * 2.0 ** top
            b.x[0] = x.to(torch.bfloat16)
            _rewrite(b)
            page = int(b.table[0, at // 16])
            assert float(b.scales[page, 0, at % 16, 1]) == 2.0 ** (top - 8)
            _check(b, f"2^{top} at {at} of {n}, lead {lead}, quiet {quiet}")
