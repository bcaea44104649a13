"""The AdamW step on the GPU, through the C ABI: bit for bit against the oracle's fp32 emulator."""

import numpy as np
import pytest
import torch

import mixture_transformers_token_gb300 as mot
from mixture_transformers_token_gb300 import workloads as W
from oracle import mot_oracle as O

from _util import bits, f64, need_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
LR, B1, B2, EPS = 3e-4, 0.9, 0.95, 1e-8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _ws():
    return torch.zeros(64, dtype=torch.uint8, device=DEV)


def _hyper(step=1, gs=1.0, lr=LR):
    return mot.mot_adamw_hyper_host(lr, B1, B2, EPS, step, gs).to(DEV)


class Case:
    """Tensors on the device, and the same on the host for the emulator."""

    def __init__(self, sizes, state="fp32", grad="fp32", p16=True, seed=1, decay=0.1):
        rng = W.rng_for(seed, 900)
        self.sizes, self.e4m3, self.decay = sizes, state == "e4m3", decay
        make = lambda n, s: (rng.standard_normal(n) * s * np.exp(rng.standard_normal(n))).astype(np.float32)  # noqa: E731
        self.p = [torch.from_numpy(make(n, 0.05)).to(DEV) for n in sizes]
        self.g = [torch.from_numpy(make(n, 1e-2)).to(DEV).to(torch.bfloat16 if grad == "bf16" else torch.float32) for n in sizes]
        self.p16 = [torch.zeros(n, dtype=torch.bfloat16, device=DEV) for n in sizes] if p16 else None
        if self.e4m3:
            self.m = [torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for n in sizes]
            self.v = [torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for n in sizes]
            self.scales = [torch.zeros((-(-n // 256), 2), device=DEV) for n in sizes]
        else:
            self.m = [torch.from_numpy(make(n, 1e-3)).to(DEV) for n in sizes]
            self.v = [torch.from_numpy(np.square(make(n, 1e-2))).to(DEV) for n in sizes]
            self.scales = None
        self.plan = mot.AdamWTensors(self.p, self.g, self.m, self.v, p16=self.p16, scales=self.scales, weight_decay=decay)

    def want(self, step, gs, seed):
        out = []
        for i in range(len(self.sizes)):
            h = np.asarray(_hyper(step, gs).cpu())[:9]
            d = self.decay if isinstance(self.decay, float) else self.decay[i]
            out.append(O.e_adamw(self.p[i].cpu().numpy(), self.g[i].float().cpu().numpy(), self.m[i].float().cpu().numpy(),
                                 self.v[i].float().cpu().numpy(), h, d, i, step, seed,
                                 self.scales[i].cpu().numpy() if self.e4m3 else None))
        return out

    def check(self, want):
        for i, w in enumerate(want):
            got = [self.p[i], self.m[i], self.v[i]] + ([self.scales[i]] if self.e4m3 else [])
            for a, b, what in zip(got, w, ("p", "m", "v", "scales")):
                a = a.float().cpu().numpy()
                same = (a == b) | (np.isnan(a) & np.isnan(b))
                assert same.all(), (what, i, int((~same).sum()), a[~same][:4], np.asarray(b)[~same][:4])
            if self.p16 is not None:
                ref = torch.from_numpy(np.asarray(w[0], np.float32)).to(torch.bfloat16)
                assert np.array_equal(bits(self.p16[i]), bits(ref)) or np.isnan(w[0]).any()


SIZES = [[1], [2, 3, 7], [8, 255, 256, 257], [2047, 2048, 2049, 100003], [5] * 130 + [300]]


@pytest.mark.parametrize("state,grad", [("fp32", "fp32"), ("fp32", "bf16"), ("e4m3", "fp32"), ("e4m3", "bf16")])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_three_steps_bit_for_bit(sizes, state, grad):
    c = Case(sizes, state, grad, seed=len(sizes))
    ws = _ws()
    for step in (1, 2, 1000003):
        want = c.want(step, 0.5, 0x1234567890ABCDEF)
        mot.mot_adamw_step(c.plan, _hyper(step, 0.5), ws, seed=0x1234567890ABCDEF)
        c.check(want)
    assert mot.mot_device_status(ws) == 0


def test_without_copies_and_decays_of_their_own():
    c = Case([300, 40, 4096], "e4m3", p16=False, decay=[0.0, 0.3, 1e-3])
    want = c.want(3, 1.0, 9)
    mot.mot_adamw_step(c.plan, _hyper(3), _ws(), seed=9)
    c.check(want)


def test_zero_small_and_loud_gradients():
    for state in ("fp32", "e4m3"):
        c = Case([256 * 9], state, seed=5)
        g = c.g[0].view(9, 256)
        g[0] = 0                      # nothing moves but by the decay
        g[1] *= 2.0 ** -60            # squares below fp32's range
        g[2] *= 2.0 ** -110
        g[3] *= 2.0 ** 60
        g[4, 3] = float("inf")
        g[5, 200] = float("nan")
        g[6] *= 2.0 ** 80             # squares above it
        g[7, 1:] = 0
        for step in (1, 2):
            want = c.want(step, 1.0, 3)
            mot.mot_adamw_step(c.plan, _hyper(step), _ws(), seed=3)
            c.check(want)
        assert torch.isfinite(c.p[0].view(9, 256)[[0, 1, 2, 3, 7, 8]]).all()


def test_a_slice_of_a_weight_and_what_is_beside_it():
    # the gen set of a [2][N][K] weight; the und set, and what lies behind, stay as they are
    w = torch.randn(2, 48, 64, device=DEV).to(torch.bfloat16)
    before = w.clone()
    n = 48 * 64 - 5
    p = w[1].float().reshape(-1)
    g, m, v = torch.randn(48, 64, device=DEV), torch.zeros(48, 64, device=DEV), torch.zeros(48, 64, device=DEV)
    plan = mot.AdamWTensors([p[:n]], [g.reshape(-1)[:n]], [m.reshape(-1)[:n]], [v.reshape(-1)[:n]], p16=[w[1].reshape(-1)[:n]])
    old = p.clone()
    mot.mot_adamw_step(plan, _hyper(), _ws())
    assert torch.equal(w[0], before[0]) and torch.equal(w[1].reshape(-1)[n:], before[1].reshape(-1)[n:])
    assert torch.equal(p[n:], old[n:]) and not m.reshape(-1)[n:].any() and not v.reshape(-1)[n:].any()
    assert torch.equal(w[1].reshape(-1)[:n], p[:n].to(torch.bfloat16)) and not torch.equal(p[:n], old[:n])


def test_eight_bit_states_follow_a_slow_average():
    # gradients whose square falls to a hundredth: the second moment follows though a step changes it by less than
    # half the distance to the next code
    n = 256 * 64
    c = Case([n], "e4m3")
    ws = _ws()
    for t in range(1, 121):
        c.g[0].copy_(torch.randn(n, device=DEV, generator=torch.Generator(DEV).manual_seed(t)) * (1.0 if t <= 40 else 0.1))
        mot.mot_adamw_step(c.plan, _hyper(t), ws, seed=1)
    v = (c.v[0].float().view(-1, 256) * c.scales[0][:, 1:]).square().mean()
    # of 1.0 after 40 steps, 0.95^80 = 0.0165 are left, and 0.01 (1 - 0.0165) come in; the mean of v / its expectation over
    # 16384 elements scatters by sqrt(2 (1 - B2) / (1 + B2) / n) = 0.0018, rounding adds about (step / sqrt(v))^2 / 6 a step
    expect = (1 - 0.95 ** 40) * 0.95 ** 80 + 0.01 * (1 - 0.95 ** 80)
    assert abs(float(v) / expect - 1) < 0.1


@pytest.mark.parametrize("word,value", [(0, -1.0), (0, float("nan")), (1, 1.0), (2, 0.0), (3, -0.1), (4, 2.0), (5, float("inf")),
                                        (6, 0.5), (7, 0.0), (8, float("inf")), (8, float("nan"))])
def test_bad_numbers_update_nothing(word, value):
    c = Case([700, 9], "e4m3")
    ws, h = _ws(), _hyper()
    mot.mot_adamw_step(c.plan, h, ws)  # states that are not zero
    before = [[t.clone() for t in x] for x in (c.p, c.p16, [y.view(torch.uint8) for y in c.m], [y.view(torch.uint8) for y in c.v], c.scales)]
    h[word] = value
    mot.mot_adamw_step(c.plan, h, ws)
    assert mot.mot_device_status(ws) == mot.DEV_BAD_HYPER
    after = (c.p, c.p16, [y.view(torch.uint8) for y in c.m], [y.view(torch.uint8) for y in c.v], c.scales)
    assert all(torch.equal(a, b) for x, y in zip(before, after) for a, b in zip(x, y))


def test_bad_step_word():
    c = Case([10])
    ws, h = _ws(), _hyper()
    for bad in (0, -1):
        h.view(torch.int32)[9] = bad
        mot.mot_adamw_step(c.plan, h, ws)
        assert mot.mot_device_status(ws) == mot.DEV_BAD_HYPER


def test_captured_steps_read_new_numbers():
    a, b = Case([5000, 77], "e4m3", seed=8), Case([5000, 77], "e4m3", seed=8)
    table = torch.stack([mot.mot_adamw_hyper_host(LR, B1, B2, EPS, t) for t in range(1, 5)]).to(DEV)
    ws, row = _ws(), torch.empty(16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    row.copy_(table[0])
    with torch.cuda.graph(graph):
        mot.mot_adamw_step(b.plan, row, ws, seed=2)
    for t in range(4):
        mot.mot_adamw_step(a.plan, table[t], ws, seed=2)
        row.copy_(table[t])
        graph.replay()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.p + a.m + a.v, b.p + b.m + b.v))


def test_two_streams():
    cases = [Case([40000, 3], "e4m3", seed=1), Case([40000, 3], "fp32", seed=2)]
    want = [c.want(1, 1.0, 4) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws, h = [_ws(), _ws()], _hyper()
    torch.cuda.synchronize()
    for c, s, w in zip(cases, streams, ws):
        mot.mot_adamw_step(c.plan, h, w, seed=4, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        c.check(w)


def test_a_tensor_past_32_bits():
    # 2^32 + 300 elements: the last ones against a small tensor with the same contents (fp32 states have no random bits)
    n, tail = 2 ** 32 + 300, 812
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    p, m, v = (torch.zeros(n, device=DEV) for _ in range(3))
    c = Case([tail], grad="bf16", p16=False)
    for big, small in ((g, c.g[0]), (p, c.p[0]), (m, c.m[0]), (v, c.v[0])):
        big[-tail:] = small
    plan = mot.AdamWTensors([p], [g], [m], [v], weight_decay=0.1)
    mot.mot_adamw_step(plan, _hyper(2), _ws())
    mot.mot_adamw_step(c.plan, _hyper(2), _ws())
    assert torch.equal(p[-tail:], c.p[0]) and torch.equal(m[-tail:], c.m[0]) and torch.equal(v[-tail:], c.v[0])
    assert not p[:4096].any()
    del g, p, m, v
    torch.cuda.empty_cache()


def test_refusals():
    c = Case([300])
    t = dict(params=c.p, grads=c.g, m=c.m, v=c.v, p16=c.p16)
    for name in t:
        for bad in ([7], [t[name][0].double()], [t[name][0].cpu()], [t[name][0][:-1]], []):
            with pytest.raises((TypeError, ValueError)):
                mot.AdamWTensors(**{**t, name: bad})
    codes = torch.zeros(300, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    for scales in (None, [torch.zeros(1, 2, device=DEV)], [None]):
        with pytest.raises((TypeError, ValueError)):
            mot.AdamWTensors(c.p, c.g, [codes], [codes.clone()], scales=scales)
    with pytest.raises((TypeError, ValueError)):
        mot.AdamWTensors(c.p, c.g, [codes], c.v, scales=[torch.zeros(2, 2, device=DEV)])
    with pytest.raises(ValueError):
        mot.mot_adamw_step(c.plan, torch.zeros(9, device=DEV), _ws())
    off = mot.AdamWTensors([c.p[0][1:]], [c.g[0][1:]], [c.m[0][1:]], [c.v[0][1:]])
    with pytest.raises(mot.MotError):
        mot.mot_adamw_step(off, _hyper(), _ws())


def test_eight_bit_states_past_32_bits(monkeypatch):
    # the last elements of more than 2^32 codes, whose random words count from the tensor's first element
    n, tail = 2 ** 32 + 2 ** 8 + 77, 2 ** 8 + 77
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GB of free memory")
    small = Case([tail], state="e4m3", grad="bf16", p16=False, seed=41)
    p, g = torch.zeros(n, device=DEV), torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    p[-tail:], g[-tail:] = small.p[0], small.g[0]
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2))
    scales = torch.zeros((-(-n // 256), 2), device=DEV)
    ws = _ws()
    mot.mot_adamw_step(mot.AdamWTensors([p], [g], [m], [v], scales=[scales], weight_decay=0.1), _hyper(3), ws, seed=9)
    assert mot.mot_device_status(ws) == 0 and (n - tail) % 256 == 0

    def words(count, tensor, step, seed):  # of the elements from n - tail on
        b = (n - tail) // 4 + np.arange(-(-count // 4), dtype=np.uint64)
        w = O.philox4x32_7((b & np.uint64(0xFFFFFFFF), b >> np.uint64(32), np.full_like(b, tensor), np.full_like(b, step)), (seed, 0))
        return np.stack(w, 1).reshape(-1)[:count].astype(np.uint32)

    monkeypatch.setattr(O, "adamw_words", words)
    zero = np.zeros(tail, np.float32)
    want = O.e_adamw(small.p[0].cpu().numpy(), small.g[0].float().cpu().numpy(), zero, zero, np.asarray(_hyper(3).cpu())[:9], 0.1, 0,
                     3, 9, np.zeros((2, 2), np.float32))
    codes = lambda t: t.view(torch.uint8)[-tail:].view(torch.float8_e4m3fn).float()  # noqa: E731
    for a, e in zip((p[-tail:], codes(m), codes(v), scales[-2:]), want):
        assert np.array_equal(a.cpu().numpy(), np.asarray(e, np.float32))
    assert not scales[:-2].any() and not p[:-tail].any()
    del p, g, m, v, scales
    torch.cuda.empty_cache()


def test_several_blocks_a_warp():
    # enough blocks that a warp takes more than one, a rest of them and of a block at each tensor's end
    c = Case([6_000_001, 300, 257 * 256 + 3, 1], state="e4m3", grad="bf16", seed=43)
    want = c.want(1, 1.0, 5)
    mot.mot_adamw_step(c.plan, _hyper(1), _ws(), seed=5)
    for i, (p, m, v, s) in enumerate(want):
        for a, e in ((c.p[i], p), (c.m[i].float(), m), (c.v[i].float(), v), (c.scales[i], s)):
            assert np.array_equal(a.cpu().numpy(), np.asarray(e, np.float32)), i
