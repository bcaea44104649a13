"""The paged key-value cache on the GPU, through the C ABI, against the oracle.

The written cache and the rows read back are compared bit for bit. A decoded output is compared with
the fp64 golden under a bound that counts each rounding:
  scores    the dot product's fp32 accumulation, at most 2 D 2^-24 sum|q||k| scale; the score times
            scale log2 e and a scale, rounded thrice: 2^-22 |s|. An error d
            of a score changes its weight by the factor e^d, and the sum of the weights by as much.
  weights   2^-20 for exp2f and the rescaling of a handful of running maxima; a weight's own rounding
            before its product with v: 2^-11 (a half, e4m3 cache) or 2^-16 (two bf16, bf16 cache).
  sums      at most 2 n 2^-24 of the sum of p|v| (n keys), once in the output and once in the sum.
  output    half a bf16 step: 2^-8 |out|.
So |got - out| <= 2^-8 |out| + E sum p|v| with the E of `_bound`.
"""

import numpy as np
import pytest
import torch

import mixture_transformers_token_gb300 as mot
from mixture_transformers_token_gb300 import workloads as W
from oracle import mot_oracle as O

from _util import assert_bitwise, f64, need_gpu

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _ws(n=64):
    return torch.zeros(n, dtype=torch.uint8, device=DEV)


def _qkv(T, Hq, Hkv, D, seed, spread=0.0):
    x = W.bf16_normal(W.rng_for(seed, 600), (T, (Hq + 2 * Hkv) * D))
    if spread:
        r = W.rng_for(seed, 601)
        x = (x.float() * torch.from_numpy(np.exp2(r.integers(-spread, spread + 1, (T, 1))).astype(np.float32))).to(
            torch.bfloat16)
    return x


def _empty_cache(n_pages, Hkv, page, D, kv, fill=0x7F):
    """A cache whose unwritten slots hold NaN (code 0x7F, bf16 0x7F7F... is finite, so bf16 gets 0x7FC0)."""
    if kv == "e4m3":
        k = torch.full((n_pages, Hkv, page, D), fill, dtype=torch.uint8, device=DEV).view(E4M3)
        return k, k.clone(), torch.full((n_pages, Hkv, page, 2), float("nan"), device=DEV)
    k = torch.full((n_pages, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    return k, k.clone(), None


def _kv(x, Hq, Hkv, D):
    """K and V of fused rows as float64 [T][Hkv][D]."""
    a = f64(x)
    T = a.shape[0]
    return (a[:, Hq * D:(Hq + Hkv) * D].reshape(T, Hkv, D), a[:, (Hq + Hkv) * D:].reshape(T, Hkv, D))


def _raw(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t.view(torch.int16)


def _slots(T, n_slots, seed, skip=0.0):
    r = W.rng_for(seed, 602)
    s = r.permutation(n_slots)[:T].astype(np.int32)
    if skip:
        s[r.random(T) < skip] = -1
    return s


def _values(t, scales=None):
    """The values that a cache stands for, float64 [slot][Hkv][D]."""
    n, h, p, d = t.shape
    x = t.to(torch.float32).cpu().numpy().astype(np.float64)
    if scales is not None:
        x = x * scales.cpu().numpy().astype(np.float64)[..., None]
    return x.transpose(0, 2, 1, 3).reshape(n * p, h, d)


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,Hq,Hkv,D,page", [(1, 4, 2, 64, 16), (2, 1, 1, 128, 16), (33, 28, 4, 128, 48),
                                             (129, 6, 3, 64, 32), (1000, 28, 4, 128, 64), (70, 2, 2, 64, 1024)])
def test_write_matches_the_oracle(T, Hq, Hkv, D, page, kv):
    n_pages = T // page + 3
    x = _qkv(T, Hq, Hkv, D, T + D, spread=9)
    slots = _slots(T, n_pages * page, T, skip=0.1 if T > 4 else 0.0)
    k, v, sc = _empty_cache(n_pages, Hkv, page, D, kv)
    before = [_raw(k).clone(), _raw(v).clone()]
    ws = _ws()
    mot.mot_kv_cache_write(x.to(DEV), torch.from_numpy(slots).to(DEV), k, v, Hq, ws, scales=sc)
    assert mot.mot_device_status(ws) == 0
    rows = np.flatnonzero(slots >= 0)
    page_of, off = slots[rows] // page, slots[rows] % page
    for i, (t, want) in enumerate(zip((k, v), _kv(x, Hq, Hkv, D))):
        got = t.to(torch.float32).cpu().numpy()[page_of, :, off].astype(np.float64)
        if kv == "bf16":
            np.testing.assert_array_equal(got, want[rows])
        else:
            y, s = O.kv_quantise(want[rows])
            np.testing.assert_array_equal(got, y)
            assert np.array_equal(np.signbit(got), np.signbit(y))
            np.testing.assert_array_equal(sc.cpu().numpy()[page_of, :, off, i].astype(np.float64), s)
        # no other slot changed
        kept = np.ones(n_pages * page, bool)
        kept[slots[rows]] = False
        now, was = (u.cpu().numpy().transpose(0, 2, 1, 3).reshape(n_pages * page, Hkv, D) for u in (_raw(t), before[i]))
        np.testing.assert_array_equal(now[kept], was[kept])
        if sc is not None:
            assert np.isnan(sc.cpu().numpy()[..., i].transpose(0, 2, 1).reshape(-1, Hkv)[kept]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_write_e4m3_borders_and_values_that_are_not_finite(D):
    Hq, Hkv, page = 1, 1, 16
    tops = [0.0, 448.0, 450.0, 446.0, 2.0 ** -55, 2.0 ** -56 * 1.75, 2.0 ** -100, 2.0 ** -133, 3.3895e38, 2.0 ** 127,
            1.75 * 2.0 ** 120, 1.7578125, 1.75, 1.0, float("inf"), float("-inf"), float("nan")]
    T = len(tops)
    x = torch.zeros((T, 3 * D))
    r = W.rng_for(4, 603)
    for i, a in enumerate(tops):
        if np.isfinite(a):
            x[i] = torch.from_numpy(r.uniform(-1, 1, 3 * D).astype(np.float32)) * a
        for c in (D + 5, 2 * D + D - 1):   # the largest of K and of V, at two places
            x[i, c] = a if i % 2 else -a
    x[3, D + 7] = -0.0
    x = x.to(torch.bfloat16)
    k, v, sc = _empty_cache(2, Hkv, page, D, "e4m3")
    ws = _ws()
    mot.mot_kv_cache_write(x.to(DEV), torch.arange(T, dtype=torch.int32, device=DEV), k, v, Hq, ws, scales=sc)
    assert mot.mot_device_status(ws) == 0
    got_s = sc.cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, 2)[:T]
    for i, (t, want) in enumerate(zip((k, v), _kv(x, Hq, Hkv, D))):
        y, s = O.kv_quantise(want[:, 0])
        got = t.to(torch.float32).cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, D)[:T]
        np.testing.assert_array_equal(got_s[:, i], s.astype(np.float32))
        np.testing.assert_array_equal(got, y)
        fine = np.isfinite(s)
        assert np.array_equal(np.signbit(got[fine]), np.signbit(y[fine]))
    # and back: a vector with a value that is not finite reads as NaN, the others as code * scale
    back = torch.zeros_like(x).to(DEV)
    mot.mot_kv_cache_read(k, v, torch.arange(T, dtype=torch.int32, device=DEV), back, Hq, ws, scales=sc)
    for i, (want, b) in enumerate(zip(_kv(x, Hq, Hkv, D), _kv(back, Hq, Hkv, D))):
        y, s = O.kv_quantise(want[:, 0])
        z = y * s[:, None]
        with np.errstate(over="ignore"):
            z = np.where(np.isnan(z), np.nan, O.bf16(np.where(np.isnan(z), 0.0, z)))
        np.testing.assert_array_equal(b[:, 0], z)


def test_bad_slots_are_reported_and_skipped():
    Hq, Hkv, D, page, n_pages = 2, 1, 64, 16, 2
    x = _qkv(5, Hq, Hkv, D, 9).to(DEV)
    slots = torch.tensor([3, 32, -2, -1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    for kv in ("bf16", "e4m3"):
        k, v, sc = _empty_cache(n_pages, Hkv, page, D, kv)
        ws = _ws()
        mot.mot_kv_cache_write(x, slots, k, v, Hq, ws, scales=sc)
        assert mot.mot_device_status(ws) == mot.DEV_BAD_PAGE
        ok = ~np.isnan(k.to(torch.float32).cpu().numpy()).reshape(n_pages * page, D).any(-1)
        assert list(np.flatnonzero(ok)) == [3]
        ws = _ws()
        y = x.clone()
        mot.mot_kv_cache_read(k, v, slots, y, Hq, ws, scales=sc)
        assert mot.mot_device_status(ws) == mot.DEV_BAD_PAGE
        assert torch.equal(y[1:], x[1:]) and torch.equal(y[0, : Hq * D], x[0, : Hq * D])
    ws = _ws()
    mot.mot_kv_cache_write(x[:1], slots[3:4].clone(), k, v, Hq, ws, scales=sc)   # -1 alone is no error
    assert mot.mot_device_status(ws) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,Hq,Hkv,D,page", [(1, 4, 2, 64, 16), (77, 28, 4, 128, 48), (513, 3, 3, 64, 16),
                                             (300, 8, 1, 128, 128)])
def test_read_returns_what_was_written(T, Hq, Hkv, D, page, kv):
    n_pages = T // page + 2
    x = _qkv(T, Hq, Hkv, D, T, spread=6).to(DEV)
    slots = _slots(T, n_pages * page, T + 1)
    k, v, sc = _empty_cache(n_pages, Hkv, page, D, kv)
    ws = _ws()
    mot.mot_kv_cache_write(x, torch.from_numpy(slots).to(DEV), k, v, Hq, ws, scales=sc)
    # read in another order, some slots twice, some rows not at all
    r = W.rng_for(T, 604)
    pick = r.integers(0, T, T + 3)
    want_slots = slots[pick].copy()
    left = r.random(T + 3) < 0.2
    want_slots[left] = -1
    y = _qkv(T + 3, Hq, Hkv, D, 5).to(DEV)
    was = y.clone()
    got = mot.mot_kv_cache_read(k, v, torch.from_numpy(want_slots).to(DEV), y, Hq, ws, scales=sc)
    assert got is y and mot.mot_device_status(ws) == 0
    assert torch.equal(y[:, : Hq * D], was[:, : Hq * D])
    lt = torch.from_numpy(left).to(DEV)
    assert torch.equal(y[lt], was[lt])
    src = x[torch.from_numpy(pick).to(DEV)][~lt]
    if kv == "bf16":
        assert torch.equal(y[~lt][:, Hq * D:], src[:, Hq * D:])
        return
    for a, b in zip(_kv(src, Hq, Hkv, D), _kv(y[~lt], Hq, Hkv, D)):
        q, s = O.kv_quantise(a)
        np.testing.assert_array_equal(b, q * s[..., None])   # 4 significant bits: exact in bf16


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

def _bound(g, lens, D, kv):
    n = np.maximum(np.asarray(lens, np.float64), 1)[:, None]
    d = 2 * D * 2.0 ** -24 * g["s_abs"] + 2.0 ** -22 * g["s_max"]
    e = 2 * np.expm1(d) + 2.0 ** -20 + (2.0 ** -11 if kv == "e4m3" else 2.0 ** -16) + 4 * n * 2.0 ** -24
    return 2.0 ** -8 * np.abs(g["out_pre"]) + e[..., None] * g["p_abs_v"] + 1e-37


class Batch:
    """Sequences in a shuffled paged cache, written by mot_kv_cache_write; free slots hold NaN and unused
    table entries hold indices out of range."""

    def __init__(self, lens, Hq, Hkv, D, kv, page, seed, q_gain=1.0, spread=0, n_pages=None):
        self.lens, self.Hq, self.Hkv, self.D, self.kv, self.page = list(lens), Hq, Hkv, D, kv, page
        pages = [-(-n // page) for n in lens]
        total = sum(pages) + 2
        self.n_pages = total if n_pages is None else n_pages
        order = W.rng_for(seed, 605).permutation(total) + (self.n_pages - total)
        width = max(max(pages), 1) + 1
        table = np.full((len(lens), width), -7, np.int32)
        table[1::2] = 2 ** 30
        at, slots = 0, []
        for r, n in enumerate(lens):
            table[r, : pages[r]] = order[at:at + pages[r]]
            at += pages[r]
            j = np.arange(n)
            slots.append(table[r, j // page].astype(np.int64) * page + j % page)
        self.k, self.v, self.scales = _empty_cache(self.n_pages, Hkv, page, D, kv)
        self.x = [_qkv(max(n, 1), Hq, Hkv, D, seed + 10 + r, spread)[:n] for r, n in enumerate(lens)]
        ws = _ws()
        if sum(lens):
            mot.mot_kv_cache_write(torch.cat(self.x).to(DEV),
                                   torch.from_numpy(np.concatenate(slots).astype(np.int32)).to(DEV), self.k, self.v, Hq,
                                   ws, scales=self.scales)
        assert mot.mot_device_status(ws) == 0
        self.q = _qkv(len(lens), Hq, Hkv, D, seed + 1)
        if q_gain != 1.0:
            self.q = (self.q.float() * q_gain).to(torch.bfloat16)
        self.q = self.q.to(DEV)
        self.table = torch.from_numpy(table).to(DEV)
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def ws(self, R=None):
        return _ws(mot.mot_paged_decode_workspace_bytes(R or len(self.lens), self.Hq, self.Hkv, self.D,
                                                        self.table.shape[1], self.page))

    def run(self, rows=None, out=None, ws=None, **kw):
        q, t, n = self.q, self.table, self.lens_t
        if rows is not None:
            i = torch.tensor(rows, device=DEV)
            q, t, n = q[i].contiguous(), t[i].contiguous(), n[i].contiguous()
        ws = self.ws(q.shape[0]) if ws is None else ws
        out = mot.mot_paged_decode_attention(q, t, n, self.k, self.v, self.Hq, ws, scales=self.scales, out=out, **kw)
        assert mot.mot_device_status(ws) == 0
        return out

    def golden(self, scale=None):
        ks, vs = [], []
        for x in self.x:
            k, v = _kv(x, self.Hq, self.Hkv, self.D)
            if self.kv == "e4m3":
                k, v = ((lambda y, s: y * s[..., None])(*O.kv_quantise(a)) if len(a) else a for a in (k, v))
            ks.append(k)
            vs.append(v)
        q = f64(self.q)[:, : self.Hq * self.D].reshape(len(self.lens), self.Hq, self.D)
        return O.g_paged_decode(q, ks, vs, self.Hq, self.Hkv, scale)

    def check(self, out, g, what):
        got = f64(out).reshape(g["out_pre"].shape)
        d, b = np.abs(got - g["out_pre"]), _bound(g, self.lens, self.D, self.kv)
        assert np.isfinite(got).all(), what
        assert np.all(d <= b), f"{what}: {np.argwhere(d > b)[:5]} worst {np.max(d / b):.2f} of the bound"
        empty = np.asarray(self.lens) == 0
        assert not got[empty].any(), what


LENS = [1, 2, 15, 16, 17, 0, 31, 32, 33, 127, 128, 129, 255, 256, 257, 0, 500, 1023]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(28, 4, 128, 16), (4, 2, 64, 16), (1, 1, 128, 48), (8, 1, 64, 32),
                                           (9, 1, 128, 64), (16, 1, 64, 128), (34, 2, 128, 16), (10, 5, 64, 1024)])
def test_decode_matches_the_golden(Hq, Hkv, D, page, kv):
    b = Batch(LENS, Hq, Hkv, D, kv, page, seed=Hq + D, spread=3)
    b.check(b.run(), b.golden(), f"{Hq}/{Hkv} heads of {D}, pages of {page}, {kv}")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,Hq,Hkv,D,page", [(4097, 28, 4, 128, 16), (20011, 7, 1, 128, 48), (9000, 4, 2, 64, 64),
                                             (6001, 24, 24, 64, 16)])
def test_decode_long_rows(n, Hq, Hkv, D, page, kv):
    b = Batch([n, n // 3, 5], Hq, Hkv, D, kv, page, seed=n)
    b.check(b.run(), b.golden(), f"{n} keys")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_sharp_and_flat_softmax(kv):
    # large queries: one key takes nearly all weight, scores far beyond exp's range; and zero queries
    for gain in (40.0, 0.0):
        b = Batch([700, 33, 1], 7, 1, 128, kv, 16, seed=3, q_gain=gain)
        b.check(b.run(), b.golden(), f"gain {gain}")
    b = Batch([300, 64], 4, 2, 64, kv, 16, seed=4)
    b.check(b.run(scale=0.5), b.golden(0.5), "scale")


def test_decode_weights_of_quiet_values_are_not_lost():
    # one loud value vector whose key gets next to no weight, among quiet ones that get all of it
    Hq, Hkv, D, page, n = 2, 1, 64, 16, 400
    b = Batch([n], Hq, Hkv, D, "e4m3", page, seed=21)
    x = b.x[0].float()
    r = W.rng_for(21, 606)
    x[:, (Hq + Hkv) * D:] *= torch.from_numpy(np.exp2(r.integers(-40, -20, (n, 1))).astype(np.float32))
    q = b.q[:, : Hq * D].float().cpu().reshape(Hq, D)
    x[200, Hq * D:(Hq + Hkv) * D] = -8 * (q[0] + q[1])   # a key against both queries
    x[200, (Hq + Hkv) * D:] = 100.0
    x[201:204, (Hq + Hkv) * D:] = 0.0                    # vectors of zeros
    b.x[0] = x.to(torch.bfloat16)
    j = np.arange(n)
    slots = b.table.cpu().numpy()[0, j // page] * page + j % page
    mot.mot_kv_cache_write(b.x[0].to(DEV), torch.from_numpy(slots.astype(np.int32)).to(DEV), b.k, b.v, Hq, _ws(),
                           scales=b.scales)
    b.check(b.run(), b.golden(), "quiet values")
    # zeros alone
    x[:, (Hq + Hkv) * D:] = 0.0
    mot.mot_kv_cache_write(x.to(torch.bfloat16).to(DEV), torch.from_numpy(slots.astype(np.int32)).to(DEV), b.k, b.v, Hq,
                           _ws(), scales=b.scales)
    assert not f64(b.run()).any()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_row_bits_do_not_depend_on_the_batch(kv):
    lens = [900, 1, 0, 77, 3000, 256, 13, 512]
    b = Batch(lens, 14, 2, 128, kv, 16, seed=31)
    all_ = b.run()
    assert_bitwise(b.run(), all_, "repeat")
    for rows in ([4], [0], [3, 5], [7, 6, 5, 4, 3, 2, 1, 0], [4] * 9):
        assert_bitwise(b.run(rows), all_[torch.tensor(rows, device=DEV)], f"rows {rows}")
    # other page indices, a wider table
    c = Batch(lens, 14, 2, 128, kv, 16, seed=31, n_pages=b.n_pages + 50)
    c.table = torch.cat([c.table, torch.full((len(lens), 300), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    assert_bitwise(c.run(), all_, "another placement")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,Hq,Hkv,D,page", [(5003, 24, 2, 128, 16), (4100, 20, 1, 64, 48), (2051, 64, 4, 64, 32),
                                             (3500, 33, 1, 128, 16)])
def test_decode_groups_of_more_than_eight_heads(n, Hq, Hkv, D, page, kv):
    lens = [n, 0, 700, 33, 1, n // 2, 512, 17] * 3
    b = Batch(lens, Hq, Hkv, D, kv, page, seed=n, spread=2)
    want = b.run()
    b.check(want, b.golden(), f"{Hq}/{Hkv} heads")
    assert_bitwise(b.run([0, 5, 2]), want[[0, 5, 2]], "a part of the batch")
    c = Batch([900, 33, 1], Hq, Hkv, D, kv, page, seed=n + 1, q_gain=40.0)
    c.check(c.run(), c.golden(), "a sharp softmax")
    # one head's NaN, in the first and in the second eight, and in the last head
    clean = f64(c.run()).reshape(3, Hq, D)
    for head in (3, 8, Hq - 1):
        was = c.q[0, head * D + 5].clone()
        c.q[0, head * D + 5] = float("nan")
        got = f64(c.run()).reshape(3, Hq, D)
        others = [h for h in range(Hq) if h != head]
        assert np.isnan(got[0, head]).all() and np.array_equal(got[0, others], clean[0, others])
        assert np.array_equal(got[1:], clean[1:])
        c.q[0, head * D + 5] = was


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_nan_and_infinity_stay_in_their_rows(kv):
    Hq, Hkv, D, page = 4, 2, 64, 16
    b = Batch([40, 50, 60, 20], Hq, Hkv, D, kv, page, seed=41)
    clean = b.run()
    # a NaN among row 1's keys (head 0), an infinity among row 2's values (head 1), a NaN in row 3's query
    bad = b.x[1].clone()
    bad[7, Hq * D + 3] = float("nan")
    bad2 = b.x[2].clone()
    bad2[59, (Hq + Hkv) * D + D + 1] = float("inf")
    t = b.table.cpu().numpy()
    for r, x in ((1, bad), (2, bad2)):
        j = np.arange(len(x))
        slots = (t[r, j // page] * page + j % page).astype(np.int32)
        mot.mot_kv_cache_write(x.to(DEV), torch.from_numpy(slots).to(DEV), b.k, b.v, Hq, _ws(), scales=b.scales)
    b.q[3, D + 2] = float("nan")
    got = b.run()
    a, c = f64(got).reshape(4, Hq, D), f64(clean).reshape(4, Hq, D)
    assert np.array_equal(a[0], c[0])
    assert np.isnan(a[1, :2]).all() and np.array_equal(a[1, 2:], c[1, 2:])
    assert np.array_equal(a[2, :2], c[2, :2]) and not np.isfinite(a[2, 2:, 1]).any()
    assert np.isnan(a[3, 1]).all() and np.array_equal(a[3, [0, 2, 3]], c[3, [0, 2, 3]])


def test_decode_reports_bad_lengths_and_pages():
    Hq, Hkv, D, page = 4, 2, 64, 16
    for kv in ("bf16", "e4m3"):
        b = Batch([40, 300, 60, 20], Hq, Hkv, D, kv, page, seed=51)
        clean = b.run()
        keep = torch.full_like(clean, -3.0)
        for lens in ([40, -1, 60, 20], [40, b.table.shape[1] * page + 1, 60, 20]):
            ws = b.ws()
            out = mot.mot_paged_decode_attention(b.q, b.table, torch.tensor(lens, dtype=torch.int32, device=DEV), b.k,
                                                 b.v, Hq, ws, scales=b.scales, out=keep.clone())
            assert mot.mot_device_status(ws) == mot.DEV_BAD_PAGE
            assert torch.equal(out[1], keep[1]) and torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]])
        for entry in (-1, b.n_pages, 2 ** 31 - 1, -2 ** 31):
            t = b.table.clone()
            t[1, 3] = entry
            ws = b.ws()
            out = mot.mot_paged_decode_attention(b.q, t, b.lens_t, b.k, b.v, Hq, ws, scales=b.scales)
            assert mot.mot_device_status(ws) == mot.DEV_BAD_PAGE
            assert torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_batches_that_begin_or_consist_of_bad_lengths(kv):
    # more rows than a producer's window holds, so that whole windows have no work
    good = [40, 700, 0, 16]
    b = Batch(good, 4, 2, 64, kv, 16, seed=52)
    want = b.run()
    n = 600
    pick = torch.cat([torch.zeros(n, dtype=torch.int64), torch.arange(4)]).to(DEV)
    q, t, lens = b.q[pick].contiguous(), b.table[pick].contiguous(), b.lens_t[pick].contiguous()
    lens[:n] = -1
    for rows in (slice(0, n + 4), slice(0, n), slice(0, 1)):
        ws = b.ws(n + 4)
        out = torch.full((len(lens[rows]), 4 * 64), -3.0, dtype=torch.bfloat16, device=DEV)
        mot.mot_paged_decode_attention(q[rows], t[rows], lens[rows], b.k, b.v, 4, ws, scales=b.scales, out=out)
        assert mot.mot_device_status(ws) == mot.DEV_BAD_PAGE
        assert (out[:n] == -3).all() and torch.equal(out[n:], want[: len(out) - len(out[:n])])


def test_decode_leaves_what_lies_around_its_outputs():
    b = Batch([70, 700, 3], 7, 1, 64, "bf16", 16, seed=61)
    want = b.run()
    n = b.ws().numel()
    big = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
    big[:64] = 0
    out = torch.full((5, 7 * 64), 9.0, dtype=torch.bfloat16, device=DEV)
    b.run(out=out[1:4], ws=big[:n])
    assert torch.equal(out[1:4], want) and (out[[0, 4]] == 9).all() and (big[n:] == 0xAB).all()


def test_decode_in_a_captured_graph_and_on_another_stream():
    b = Batch([600, 1, 30, 2000], 28, 4, 128, "e4m3", 16, seed=71)
    want = b.run()
    short = torch.tensor([17, 0, 30, 1999], dtype=torch.int32, device=DEV)
    full = b.lens_t.clone()
    b.lens_t.copy_(short)
    want_short = b.run()
    b.lens_t.copy_(full)
    ws, out = b.ws(), torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mot.mot_paged_decode_attention(b.q, b.table, b.lens_t, b.k, b.v, b.Hq, ws, scales=b.scales, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    mot.mot_paged_decode_attention(b.q, b.table, b.lens_t, b.k, b.v, b.Hq, ws, scales=b.scales, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):   # two calls that share a workspace
            mot.mot_paged_decode_attention(b.q, b.table, b.lens_t, b.k, b.v, b.Hq, ws, scales=b.scales, out=out)
    for lens, w in ((full, want), (short, want_short), (full, want)):
        b.lens_t.copy_(lens)
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert mot.mot_device_status(ws) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_beyond_32_bits(kv):
    # the last pages of a cache of more than 2^32 bytes of K (2^31 elements in bf16)
    Hq, Hkv, D, page = 8, 8, 128, 64
    n_pages = (1 << 32) // (Hkv * page * D * (1 if kv == "e4m3" else 2)) + 40
    b = Batch([700, 150], Hq, Hkv, D, kv, page, seed=81, n_pages=n_pages)
    assert int(b.table[0, 0]) * Hkv * page * D * (1 if kv == "e4m3" else 2) > (1 << 32) - (1 << 24)
    b.check(b.run(), b.golden(), "high pages")
    y = torch.zeros_like(b.q[:1])
    slot = int(b.table[0, 1]) * page + 3
    mot.mot_kv_cache_read(b.k, b.v, torch.tensor([slot], dtype=torch.int32, device=DEV), y, Hq, _ws(), scales=b.scales)
    for a, c in zip(_kv(b.x[0][page + 3: page + 4], Hq, Hkv, D), _kv(y, Hq, Hkv, D)):
        if kv == "e4m3":
            q, s = O.kv_quantise(a)
            a = q * s[..., None]
        np.testing.assert_array_equal(c, a)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_many_rows(kv):
    # more rows than the walk holds at a time, more items a CTA than descriptors in flight; bad rows between
    r = W.rng_for(7, 607)
    lens = [int(n) for n in r.integers(0, 1400, 300)]
    lens[255], lens[256], lens[299] = 1399, 0, 1
    b = Batch(lens, 8, 4, 64, kv, 16, seed=101)
    out = b.run()
    b.check(out, b.golden(), "300 rows")
    bad = b.lens_t.clone()
    at = torch.tensor([0, 31, 32, 100, 255, 256, 299], device=DEV)
    bad[at] = torch.tensor([-1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, -1, -5, 2 ** 30], dtype=torch.int32, device=DEV)
    ws, keep = b.ws(), torch.full_like(out, 2.0)
    got = mot.mot_paged_decode_attention(b.q, b.table, bad, b.k, b.v, 8, ws, scales=b.scales, out=keep.clone())
    assert mot.mot_device_status(ws) == mot.DEV_BAD_PAGE
    fine = torch.ones(300, dtype=torch.bool, device=DEV)
    fine[at] = False
    assert torch.equal(got[fine], out[fine]) and torch.equal(got[~fine], keep[~fine])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_row_bits_do_not_depend_on_the_table_width_or_the_join(kv):
    # few rows take one form of the join, many the other (also with more than 32 ranges); so do narrow tables
    b = Batch([6000, 300, 40000, 1500], 7, 1, 128, kv, 16, seed=111)
    want = b.run()
    b.check(want, b.golden(), "few rows")
    rows = [0, 1, 2, 3] * 90
    assert_bitwise(b.run(rows), want[torch.tensor(rows, device=DEV)], "many rows")
    short = b.table
    b.table = torch.cat([b.table, torch.full((4, 3000), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    assert_bitwise(b.run(), want, "wide table")
    assert_bitwise(b.run(rows), want[torch.tensor(rows, device=DEV)], "wide table, many rows")
    b.table = short[:, : 1500 // 16 + 1].contiguous()
    assert_bitwise(b.run([3, 1]), want[[3, 1]], "narrow table")


def test_parts_of_longer_index_arrays():
    # slots, tables and lengths that start inside longer tensors, on 4-byte boundaries
    b = Batch([70, 33, 200, 16, 90], 4, 2, 64, "e4m3", 16, seed=115)
    want = b.run()
    width = b.table.shape[1]
    lens = torch.cat([torch.zeros(3, dtype=torch.int32, device=DEV), b.lens_t])[3:]
    table = torch.cat([torch.full((1,), -5, dtype=torch.int32, device=DEV), b.table.reshape(-1)])[1:].reshape(5, width)
    assert lens.data_ptr() % 16 and table.data_ptr() % 16
    ws = b.ws()
    got = mot.mot_paged_decode_attention(b.q, table, lens, b.k, b.v, 4, ws, scales=b.scales)
    assert mot.mot_device_status(ws) == 0
    assert_bitwise(got, want, "shifted arrays")
    slots = torch.arange(9, dtype=torch.int32, device=DEV)
    y = mot.mot_kv_cache_read(b.k, b.v, slots[1:], b.q.new_zeros((8, b.q.shape[1])), 4, ws, scales=b.scales)
    z = mot.mot_kv_cache_read(b.k, b.v, slots[1:].clone(), b.q.new_zeros((8, b.q.shape[1])), 4, ws, scales=b.scales)
    assert_bitwise(y, z, "shifted slots")


def test_decode_scales_that_are_no_powers_of_two():
    b = Batch([333, 40, 1], 14, 2, 128, "e4m3", 16, seed=121)
    r = W.rng_for(8, 608)
    f = torch.from_numpy(np.exp2(r.uniform(-6, 6, tuple(b.scales.shape))).astype(np.float32)).to(DEV)
    b.scales *= f
    n_pages, Hkv, page, _ = b.scales.shape
    k, v = (_values(t, b.scales[..., i]) for i, t in enumerate((b.k, b.v)))
    tab = b.table.cpu().numpy()
    rows = [[tab[i, j // page] * page + j % page for j in range(n)] for i, n in enumerate(b.lens)]
    q = f64(b.q)[:, : b.Hq * b.D].reshape(len(b.lens), b.Hq, b.D)
    g = O.g_paged_decode(q, [k[x] for x in rows], [v[x] for x in rows], b.Hq, b.Hkv)
    b.check(b.run(), g, "scales")


def test_decode_on_two_streams_at_once():
    a, b = Batch([3000, 50, 700], 28, 4, 128, "e4m3", 32, seed=131), Batch([900] * 9, 4, 2, 64, "bf16", 16, seed=132)
    want_a, want_b = a.run(), b.run()
    wa, wb, oa, ob = a.ws(), b.ws(), torch.empty_like(want_a), torch.empty_like(want_b)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        mot.mot_paged_decode_attention(a.q, a.table, a.lens_t, a.k, a.v, a.Hq, wa, scales=a.scales, out=oa, stream=sa)
        mot.mot_paged_decode_attention(b.q, b.table, b.lens_t, b.k, b.v, b.Hq, wb, out=ob, stream=sb)
    torch.cuda.synchronize()
    assert torch.equal(oa, want_a) and torch.equal(ob, want_b)
    assert mot.mot_device_status(wa) == 0 and mot.mot_device_status(wb) == 0


def test_write_and_read_in_a_captured_graph():
    Hq, Hkv, D, page, T = 4, 2, 64, 16, 40
    x = _qkv(T, Hq, Hkv, D, 141).to(DEV)
    slots = torch.from_numpy(_slots(T, 64, 142)).to(DEV)
    k, v, sc = _empty_cache(4, Hkv, page, D, "e4m3")
    ws, y = _ws(), torch.zeros_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mot.mot_kv_cache_write(x, slots, k, v, Hq, ws, scales=sc)
        mot.mot_kv_cache_read(k, v, slots, y, Hq, ws, scales=sc)
    for seed in (143, 144):
        x.copy_(_qkv(T, Hq, Hkv, D, seed).to(DEV))
        slots.copy_(torch.from_numpy(_slots(T, 64, seed)).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(_kv(x, Hq, Hkv, D), _kv(y, Hq, Hkv, D)):
            q, s = O.kv_quantise(a)
            np.testing.assert_array_equal(b, q * s[..., None])
    assert mot.mot_device_status(ws) == 0


# ---------------------------------------------------------------------------
# the calls together, as a server makes them
# ---------------------------------------------------------------------------

def test_projection_cache_and_decode_together():
    # QKV projection of prompts -> cache; then three decoding steps, each projecting one row a sequence,
    # writing it and attending; every step's output against the golden over all rows projected so far
    s, inp = W.tiny_layer(seed=5)
    d = {k: v.to(DEV) for k, v in inp.items() if isinstance(v, torch.Tensor)}
    prompts, page = [23, 0, 17], 16
    Hq, Hkv, D = s.Hq, s.Hkv, s.D
    k, v, sc = _empty_cache(9, Hkv, page, D, "bf16")
    table = torch.tensor([[8, 1, 4], [0, 3, 2], [5, 7, 6]], dtype=torch.int32, device=DEV)
    tab = table.cpu().numpy()
    cs = mot.mot_rope_table_fill_host(s.theta, D, 128).to(DEV)
    seen = [[] for _ in prompts]

    def project(x, mod, pos):
        ws = mot.mot_route_plan(mod)
        return mot.mot_routed_qkv_norm_rope(x, d["w_qkv"], d["q_norm"], d["k_norm"], pos, cs, Hq, Hkv, D, s.eps, ws)

    def append(rows, seq_of, pos_of):
        slots = [int(tab[q, p // page]) * page + p % page for q, p in zip(seq_of, pos_of)]
        mot.mot_kv_cache_write(rows, torch.tensor(slots, dtype=torch.int32, device=DEV), k, v, Hq, ws)
        for i, q in enumerate(seq_of):
            seen[q].append(rows[i].cpu())

    ws = _ws(mot.mot_paged_decode_workspace_bytes(3, Hq, Hkv, D, 3, page))
    seq_of = [q for q, n in enumerate(prompts) for _ in range(n)]
    pos_of = [p for n in prompts for p in range(n)]
    T = len(seq_of)
    rows = project(d["x"][:T].contiguous(), d["mod"][:T].contiguous(),
                   torch.tensor(pos_of, dtype=torch.int32, device=DEV))
    append(rows, seq_of, pos_of)
    for step in range(3):
        pos = [n + step for n in prompts]
        x = W.bf16_normal(W.rng_for(5, 700 + step), (3, s.H)).to(DEV)
        rows = project(x, torch.zeros(3, dtype=torch.uint8, device=DEV),
                       torch.tensor(pos, dtype=torch.int32, device=DEV))
        append(rows, [0, 1, 2], pos)
        lens = [p + 1 for p in pos]
        out = mot.mot_paged_decode_attention(rows, table, torch.tensor(lens, dtype=torch.int32, device=DEV), k, v, Hq, ws)
        assert mot.mot_device_status(ws) == 0
        kv = [_kv(torch.stack(x), Hq, Hkv, D) for x in seen]
        g = O.g_paged_decode(f64(rows)[:, : Hq * D].reshape(3, Hq, D), [a for a, _ in kv], [b for _, b in kv], Hq, Hkv)
        assert np.all(np.abs(f64(out).reshape(3, Hq, D) - g["out_pre"]) <= _bound(g, lens, D, "bf16"))


def test_joint_attention_over_a_prefix_read_from_the_cache():
    # prefill in two chunks: the second chunk's joint attention over a prefix that comes back from a bf16
    # cache gives the same bits as over the rows themselves
    Hq, Hkv, D, n, pre, page = 4, 2, 128, 300, 211, 32
    x = _qkv(n, Hq, Hkv, D, 91).to(DEV)
    seqs = torch.tensor([[pre, 0, n - pre, n, 40]], dtype=torch.int32, device=DEV)
    ws = _ws()
    want = mot.mot_joint_attention(x, seqs, Hq, Hkv, D, ws)
    k, v, _ = _empty_cache(10, Hkv, page, D, "bf16")
    slots = torch.from_numpy(_slots(pre, 320, 92)).to(DEV)
    mot.mot_kv_cache_write(x[:pre], slots, k, v, Hq, ws)
    y = torch.zeros_like(x)
    y[pre:] = x[pre:]
    mot.mot_kv_cache_read(k, v, slots, y[:pre], Hq, ws)
    got = mot.mot_joint_attention(y, seqs, Hq, Hkv, D, ws)
    assert mot.mot_device_status(ws) == 0
    assert_bitwise(got[pre:], want[pre:], "second chunk")


def test_binding_refuses_wrong_tensors():
    b = Batch([40], 4, 2, 64, "e4m3", 16, seed=95)
    slots = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        mot.mot_kv_cache_write(b.q, slots, b.k, b.v, 4, _ws())                        # no scales
    with pytest.raises(ValueError):
        mot.mot_kv_cache_write(b.q, slots, b.k, b.v, 6, _ws(), scales=b.scales)       # qkv's width
    with pytest.raises(ValueError):
        mot.mot_kv_cache_read(b.k, b.v, slots, b.q, 4, _ws(), scales=b.scales[:1])
    with pytest.raises(TypeError):
        mot.mot_kv_cache_read(b.k, b.v, slots.long(), b.q, 4, _ws(), scales=b.scales)
    with pytest.raises(TypeError):
        mot.mot_kv_cache_read(b.k, b.v.to(torch.bfloat16), slots, b.q, 4, _ws(), scales=b.scales)
    with pytest.raises(ValueError):
        mot.mot_paged_decode_attention(b.q, b.table, b.lens_t[:0], b.k, b.v, 4, b.ws(), scales=b.scales)
    with pytest.raises(ValueError):
        mot.mot_paged_decode_attention(b.q, b.table.t(), b.lens_t, b.k, b.v, 4, b.ws(), scales=b.scales)
    with pytest.raises(mot.MotError):
        mot.mot_paged_decode_attention(b.q, b.table, b.lens_t, b.k, b.v, 4, _ws(48), scales=b.scales)
