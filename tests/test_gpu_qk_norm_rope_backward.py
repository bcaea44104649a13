"""The gradient through the QKV projection's epilogue on the GPU, through the C ABI, against the fp64 oracle within its
counted bound."""

import numpy as np
import pytest
import torch

import mixture_transformers_token_gb300 as mot
from mixture_transformers_token_gb300 import workloads as W
from oracle import mot_oracle as O

from _util import assert_bitwise, f64, need_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS, THETA = 1e-6, 1e6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _case(T, Hq, Hkv, D, profile, gen=0.4, seed=1, P=None):
    r = W.rng_for(seed, 800)
    N, P = (Hq + 2 * Hkv) * D, P or 2 * T
    c = {"x": W.bf16_normal(r, (T, N)).to(DEV), "d": W.bf16_normal(r, (T, N)).to(DEV),
         "qw": W.bf16_normal(r, (2, D), mean=1.0, std=0.1).to(DEV), "kw": W.bf16_normal(r, (2, D), mean=1.0, std=0.1).to(DEV),
         "mod": W.modality_bernoulli(r, T, gen).to(DEV)}
    c["pos"] = torch.from_numpy(r.integers(0, P, T).astype(np.int32)).to(DEV)
    fill = mot.mot_rope_table_fill_host if profile == "bf16" else mot.mot_rope_table_fill_host_fp32
    c["cs"] = fill(THETA, D, P).to(DEV)
    c["ws"] = mot.mot_route_plan(c["mod"])
    c["heads"] = (Hq, Hkv, D)
    return c


def _run(c, **kw):
    return mot.mot_qk_norm_rope_backward(c["d"], c["x"], c["qw"], c["kw"], c["pos"], c["cs"], *c["heads"], EPS, c["ws"], **kw)


def _golden(c):
    cs = f64(c["cs"])[c["pos"].cpu().numpy()]
    return O.g_qk_norm_rope_backward(f64(c["d"]), f64(c["x"]), f64(c["qw"]), f64(c["kw"]), cs[..., 0], cs[..., 1],
                                     c["mod"].cpu().numpy(), *c["heads"], EPS)


def _check(c, dx, dw):
    g = _golden(c)
    assert np.all(np.abs(f64(dx) - g["dx"]) <= g["err_dx"] + 1e-38)
    if dw is not None:
        assert np.all(np.abs(dw.double().cpu().numpy() - g["dw"]) <= g["err_dw"] + 1e-38)
    return g


@pytest.mark.parametrize("profile", ["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 4, 2, 64), (2, 1, 1, 128), (64, 4, 2, 64), (609, 28, 4, 128), (1300, 5, 3, 64),
                                        (77, 33, 3, 128), (40, 96, 8, 128), (257, 7, 1, 128)])
def test_within_the_counted_bound(T, Hq, Hkv, D, profile):
    c = _case(T, Hq, Hkv, D, profile, seed=T)
    dx, dw = _run(c)
    _check(c, dx, dw)
    dx2, dw2 = _run(c)
    assert_bitwise(dx, dx2, "dx again")
    assert torch.equal(dw, dw2) and mot.mot_device_status(c["ws"]) == 0


@pytest.mark.parametrize("gen", [0.0, 1.0])
def test_one_weight_set_alone(gen):
    c = _case(700, 4, 2, 64, "bf16", gen=gen)
    dx, dw = _run(c)
    _check(c, dx, dw)
    assert not dw[:, 1 - int(gen)].any()


def test_in_place_and_without_weight_gradients():
    c = _case(300, 7, 1, 128, "fp32")
    dx, dw = _run(c)
    same, none = _run(c, sets=0)
    assert none is None
    assert_bitwise(dx, same, "without weight gradients")
    d = c["d"].clone()
    c["d"] = d
    got, dw3 = _run(c, dx=d)
    assert got is d and torch.equal(dw, dw3)
    assert_bitwise(dx, d, "in place")


def test_sets_leave_the_other_rows():
    c = _case(300, 4, 2, 64, "bf16")
    _, both = _run(c)
    for sets, i in ((mot.SET_UND, 0), (mot.SET_GEN, 1)):
        dw = torch.full((2, 2, 64), 9.0, device=DEV)
        _run(c, sets=sets, dw=dw)
        assert torch.equal(dw[:, i], both[:, i]) and torch.all(dw[:, 1 - i] == 9.0)


def test_small_and_zero_heads():
    # heads where eps decides the norm, a head of zeros, loud heads
    c = _case(64, 4, 2, 64, "bf16")
    c["x"][:10] *= 1e-3
    c["x"][10] = 0
    c["x"][11] *= 2.0 ** 40
    dx, dw = _run(c)
    _check(c, dx, dw)


def test_rows_do_not_depend_on_the_pack():
    c = _case(500, 4, 2, 64, "bf16", seed=3)
    dx, _ = _run(c)
    for n in (1, 63, 200):
        part = {**c, "d": c["d"][:n].contiguous(), "x": c["x"][:n].contiguous(), "pos": c["pos"][:n].contiguous(),
                "ws": mot.mot_route_plan(c["mod"][:n].contiguous())}
        assert_bitwise(_run(part)[0], dx[:n], f"{n} rows")


def test_offsets_past_32_bits():
    # rows whose elements lie past 2^31 values: the last rows against a small call
    Hq, Hkv, D, T = 96, 8, 128, 152000
    N = (Hq + 2 * Hkv) * D
    assert T * N > 2 ** 31
    d = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    small = _case(50, Hq, Hkv, D, "bf16", seed=4)
    x = torch.ones((T, N), dtype=torch.bfloat16, device=DEV)
    d[-50:], x[-50:] = small["d"], small["x"]
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    pos[-50:] = small["pos"]
    mod = torch.zeros(T, dtype=torch.uint8, device=DEV)
    mod[-50:] = small["mod"]
    c = {**small, "d": d, "x": x, "pos": pos, "ws": mot.mot_route_plan(mod)}
    dx, _ = _run(c, dx=d)
    assert_bitwise(dx[-50:], _run(small)[0], "the last rows")


def test_bad_positions_and_plans():
    c = _case(30, 4, 2, 64, "bf16")
    want = _run(c)[0]
    at0 = c["pos"].clone()
    at0[[3, 9]] = 0
    c["pos"] = at0
    zero = _run(c)[0]
    bad = at0.clone()
    bad[3], bad[9] = -1, c["cs"].shape[0]
    c["pos"] = bad
    got = _run(c)[0]
    assert mot.mot_device_status(c["ws"]) == mot.DEV_BAD_POSITION
    assert_bitwise(got, zero, "bad positions are taken as 0")
    assert not torch.equal(want, zero)
    # a plan of another T: nothing is written
    other = mot.mot_route_plan(torch.zeros(31, dtype=torch.uint8, device=DEV))
    dx, dw = torch.full_like(c["d"], 7.0), torch.full((2, 2, 64), 7.0, device=DEV)
    _run({**c, "ws": other}, dx=dx, dw=dw)
    assert mot.mot_device_status(other) == mot.DEV_PLAN_MISMATCH and torch.all(dx == 7.0) and torch.all(dw == 7.0)


def test_captured_and_on_two_streams():
    a, b = _case(200, 4, 2, 64, "bf16", seed=6), _case(200, 4, 2, 64, "fp32", seed=7)
    wa, wb = _run(a), _run(b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    n = mot.mot_qk_norm_rope_backward_workspace_bytes(200, 64)
    bufs = [dict(dx=torch.empty_like(a["d"]), dw=torch.empty((2, 2, 64), device=DEV),
                 scratch=torch.empty(n, dtype=torch.uint8, device=DEV)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, o in ((a, streams[0], bufs[0]), (b, streams[1], bufs[1])):
            _run(c, stream=s, **o)
    torch.cuda.synchronize()
    for w, o in ((wa, bufs[0]), (wb, bufs[1])):
        assert_bitwise(w[0], o["dx"], "dx")
        assert torch.equal(w[1], o["dw"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(a, **bufs[0])
    d = a["d"].clone()
    a["d"].mul_(2)  # exact: the gradient doubles
    graph.replay()
    assert torch.equal(bufs[0]["dw"], wa[1] * 2)
    a["d"].copy_(d)
    graph.replay()
    assert_bitwise(bufs[0]["dx"], wa[0], "replayed")


def test_refusals():
    c = _case(30, 4, 2, 64, "bf16")
    names = {"d_out": "d", "x": "x", "q_norm_w": "qw", "k_norm_w": "kw", "pos": "pos", "rope_cs": "cs", "ws": "ws"}
    for name, key in names.items():
        for bad in (7, c[key].double(), c[key].cpu(), c[key].unsqueeze(0)):
            with pytest.raises((TypeError, ValueError), match=name):
                _run({**c, key: bad})
    for kw in (dict(dx=c["x"][:-1].contiguous()), dict(dw=torch.zeros(2, 64, device=DEV)), dict(sets=0, dw=torch.zeros(2, 2, 64, device=DEV))):
        with pytest.raises(ValueError):
            _run(c, **kw)
    for kw in (dict(sets=4), dict(scratch=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(mot.MotError):
            _run(c, **kw)
