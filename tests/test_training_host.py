"""The training step's operators without a GPU: pins of the oracle's gradients and update, the numbers of an optimizer step,
and the entry points' refusals (made before any CUDA call)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import mixture_transformers_token_gb300 as mot
from mixture_transformers_token_gb300 import build as mot_build
from oracle import mot_oracle as O

MOT_ERR_NULL, MOT_ERR_ALIGN, MOT_ERR_GEOMETRY, MOT_ERR_WORKSPACE, MOT_ERR_ARG = 1, 2, 3, 5, 8
A, B, C, E, F, G, H = (n << 20 for n in (1, 2, 3, 5, 6, 7, 8))  # fake, aligned, not NULL
MIS = (4 << 20) + 8


@pytest.fixture(scope="module")
def lib():
    mot_build.build()
    return mot.load_library()


# ---------------------------------------------------------------------------
# the oracle's gradients against differences of its forwards
# ---------------------------------------------------------------------------

def test_attention_gradient_against_differences():
    rng = np.random.default_rng(1)
    Hq, Hkv, D = 4, 2, 8
    # a prompt, latents over the prompt's keys and their own, latents over the prompt's keys alone, rows of nobody
    seqs = [(0, 0, 5, 5, 5), (8, 3, 4, 9, 2), (12, 0, 3, 5, 0)]
    T = 17
    qkv, dout = rng.standard_normal((T, (Hq + 2 * Hkv) * D)), rng.standard_normal((T, Hq * D))
    out = O.g_joint_attention(qkv, seqs, Hq, Hkv, D)["out_pre"]
    lse, _ = O.g_attention_lse(qkv, seqs, Hq, Hkv, D)
    g = O.g_joint_attention_backward(dout, qkv, out, lse, seqs, Hq, Hkv, D)
    for r, c in rng.integers(0, [T, qkv.shape[1]], (150, 2)):
        step = np.zeros_like(qkv)
        step[r, c] = 1e-5
        f = [float((O.g_joint_attention(qkv + s * step, seqs, Hq, Hkv, D)["out_pre"] * dout).sum()) for s in (1, -1)]
        assert abs((f[0] - f[1]) / 2e-5 - g["dqkv"][r, c]) <= 1e-7
    assert not g["dqkv"][~g["written"]].any() and not g["written"][15:].any() and not g["written"][12:15, Hq * D:].any()


def test_lse_is_the_softmax_sum():
    rng = np.random.default_rng(2)
    qkv = rng.standard_normal((6, 3 * 8))
    lse, _ = O.g_attention_lse(qkv, [(1, 0, 4, 5, 2)], 1, 1, 8, scale=0.7)
    for i, n in ((0, 2), (1, 3), (2, 5), (3, 5)):
        want = math.log(sum(math.exp(0.7 * float(qkv[1 + i, :8] @ qkv[j, 8:16])) for j in range(n)))
        assert abs(lse[0, 1 + i] - want) <= 1e-12


@pytest.mark.parametrize("profile", ["bf16", "fp32"])
def test_qk_norm_rope_gradient_against_differences(profile):
    rng = np.random.default_rng(3)
    T, Hq, Hkv, D, eps, theta = 5, 2, 1, 8, 1e-3, 100.0
    mod, pos = np.array([0, 1, 1, 0, 1]), np.arange(T) * 3
    x, d = rng.standard_normal((T, 4 * D)), rng.standard_normal((T, 4 * D))
    qn, kn = 1 + 0.1 * rng.standard_normal((2, D)), 1 + 0.1 * rng.standard_normal((2, D))
    c, s = (O.rope_cos_sin if profile == "bf16" else O.rope_cos_sin_f32)(theta, D, pos)
    c, s = np.asarray(c, np.float64), np.asarray(s, np.float64)

    def forward(x, qn, kn):
        y = x.copy()
        for h in range(Hq + Hkv):
            w = (qn if h < Hq else kn)[mod]
            u = x[:, h * D:(h + 1) * D]
            u = u / np.sqrt((u * u).mean(1, keepdims=True) + float(np.float32(eps))) * w
            y[:, h * D:h * D + D // 2] = u[:, :D // 2] * c - u[:, D // 2:] * s
            y[:, h * D + D // 2:(h + 1) * D] = u[:, D // 2:] * c + u[:, :D // 2] * s
        return float((y * d).sum())

    g = O.g_qk_norm_rope_backward(d, x, qn, kn, c, s, mod, Hq, Hkv, D, eps)
    for a, grad, put in ((x, g["dx"], lambda z: (z, qn, kn)), (qn, g["dw"][0], lambda z: (x, z, kn)),
                         (kn, g["dw"][1], lambda z: (x, qn, z))):
        for r, col in np.ndindex(a.shape):
            step = np.zeros_like(a)
            step[r, col] = 1e-5
            diff = (forward(*put(a + step)) - forward(*put(a - step))) / 2e-5
            assert abs(diff - grad[r, col]) <= 1e-6


# ---------------------------------------------------------------------------
# the optimizer
# ---------------------------------------------------------------------------

def test_adamw_emulator_against_torch():
    rng = np.random.default_rng(4)
    n, lr, b1, b2, eps, wd = 700, 1e-3, 0.9, 0.95, 1e-8, 0.1
    w = torch.tensor(rng.standard_normal(n), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([w], lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd)
    p, m, v = w.detach().numpy().astype(np.float32), np.zeros(n, np.float32), np.zeros(n, np.float32)
    for t in range(1, 6):
        g = rng.standard_normal(n).astype(np.float32)
        w.grad = torch.from_numpy(g).double()
        opt.step()
        p, m, v = O.e_adamw(p, g * 4, m, v, O.adamw_hyper(lr, b1, b2, eps, t, 0.25), wd)
        # a step moves p by at most lr (about 1.3: |m| / sqrt(v) corrected) and rounds it once, to 2^-24 of |p| < 4
        assert np.abs(p - w.detach().numpy()).max() <= t * (2.0 ** -22 + 64 * 2.0 ** -24 * lr)


def test_philox_words():
    # the known answers that the generator's authors publish for seven rounds
    assert [int(w) for w in O.philox4x32_7((0, 0, 0, 0), (0, 0))] == [0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48]
    f = 0xFFFFFFFF
    assert [int(w) for w in O.philox4x32_7((f, f, f, f), (f, f))] == [0x5207DDC2, 0x45165E59, 0x4D8EE751, 0x8C52F662]
    w = O.adamw_words(11, 3, 5, 0x123456789ABCDEF0)
    b = O.philox4x32_7((2, 0, 3, 5), (0x9ABCDEF0, 0x12345678))
    assert w.size == 11 and [int(i) for i in w[8:]] == [int(i) for i in b[:3]]
    u = O.adamw_words(1 << 16, 0, 1, 0) & 0xFFFF
    assert abs(float(u.mean()) - 32767.5) < 5 * 18918 / 256  # five standard errors of a uniform's mean


def test_quantiser_is_unbiased_and_takes_neighbours():
    rng = np.random.default_rng(6)
    x = (rng.standard_normal(256) * np.exp(2 * rng.standard_normal(256))).astype(np.float32)
    x[0] = 0
    values = O.e4m3_values()
    total = np.zeros(256)
    for k in range(0, 65536, 64):  # every 1024th of a step
        z, s = O.adamw_quantise(x, np.full(256, k))
        total += z
        y = np.abs(x.astype(np.float64)) * (448.0 / float(np.abs(x).max()))
        near = np.searchsorted(values, y * (1 - 1e-6))
        assert np.all((np.abs(z) <= values[np.minimum(near + 1, 126)]) & (np.abs(z) >= values[np.maximum(near - 1, 0)]))
        assert np.all(np.isin(np.abs(z), values)) and s[0] == np.abs(x).max() * (np.float32(1) / np.float32(448))
    step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3), 2.0 ** -9)
    assert np.all(np.abs(np.sign(x) * total / 1024 - y) <= step / 1024 + 1e-6 * y)
    z, s = O.adamw_quantise(np.array([1e-9, 448.0, 0.0], np.float32), np.zeros(3), keep_positive=True)
    assert z.tolist() == [2.0 ** -9, 448.0, 0.0] and abs(s[0] - 1) <= 2.0 ** -23
    z, s = O.adamw_quantise(np.full(3, 2.0 ** -101, np.float32), np.full(3, 65535), keep_positive=True)
    assert not z.any() and s[0] == 0
    assert np.isnan(O.adamw_quantise(np.array([1.0, np.inf], np.float32), np.zeros(2))[1][0])


def test_hyper_row(lib):
    row = mot.mot_adamw_hyper_host(3e-4, 0.9, 0.95, 1e-8, 12, grad_scale=0.5)
    assert row.shape == (16,) and row.view(torch.int32)[9] == 12 and not row.view(torch.int32)[10:].any()
    want = O.adamw_hyper(3e-4, 0.9, 0.95, 1e-8, 12, 0.5)
    # both powers are within an ulp of double: the fp32 roundings agree but beside a tie
    assert np.all(np.abs(row[:9].numpy() - want) <= 2.0 ** -23 * np.abs(want))
    assert mot.mot_adamw_hyper_host(0.0, 0.0, 0.0, 1e-8, 1)[5] == 0
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(lr=1e39), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
                dict(beta2=1 - 1e-12), dict(eps=0.0), dict(eps=1e-60), dict(eps=float("inf")), dict(step=0), dict(step=2 ** 31),
                dict(grad_scale=float("inf")), dict(grad_scale=float("nan"))):
        with pytest.raises(mot.MotError) as e:
            mot.mot_adamw_hyper_host(**{**dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1), **bad})
        assert e.value.status == MOT_ERR_ARG
    assert lib.mot_adamw_hyper_host(1e-3, 0.9, 0.95, 1e-8, 1.0, 1, None) == MOT_ERR_NULL


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def _attention_calls(lib):
    base = dict(dout=A, qkv=B, out=C, lse=E, T=64, Hq=4, Hkv=2, D=64, seqs=F, n=2, scale=0.125, ws=G, wsb=1 << 30, dqkv=H)

    def lse(**kw):
        a = {**base, **kw}
        return lib.mot_joint_attention_lse(a["qkv"], a["T"], a["Hq"], a["Hkv"], a["D"], a["seqs"], a["n"], a["scale"],
                                           a["ws"], a["wsb"], a["out"], a["lse"], None)

    def back(**kw):
        a = {**base, **kw}
        return lib.mot_joint_attention_backward(a["dout"], a["qkv"], a["out"], a["lse"], a["T"], a["Hq"], a["Hkv"], a["D"],
                                                a["seqs"], a["n"], a["scale"], a["ws"], a["wsb"], a["dqkv"], None)

    return lse, back


def test_attention_calls_reject(lib):
    lse, back = _attention_calls(lib)
    for f, names in ((lse, ("qkv", "out", "lse", "seqs", "ws")), (back, ("dout", "qkv", "out", "lse", "seqs", "ws", "dqkv"))):
        for name in names:
            assert f(**{name: None}) == MOT_ERR_NULL, name
            assert f(**{name: MIS}) == MOT_ERR_ALIGN, name
        for bad in (dict(T=0), dict(T=(1 << 24) + 1), dict(D=96), dict(Hq=3), dict(Hkv=0), dict(Hq=0), dict(Hq=1025, Hkv=1),
                    dict(n=0), dict(n=-1)):
            assert f(**bad) == MOT_ERR_GEOMETRY, bad
        for scale in (0.0, -1.0, float("nan"), float("inf")):
            assert f(scale=scale) == MOT_ERR_ARG
        assert f(wsb=63) == MOT_ERR_WORKSPACE
        assert f() not in (0, MOT_ERR_NULL, MOT_ERR_ALIGN, MOT_ERR_GEOMETRY, MOT_ERR_ARG, MOT_ERR_WORKSPACE)  # the device
    for scale in (2.0 ** -101, 2.0 ** 100):
        assert back(scale=scale) == MOT_ERR_ARG
    need = lib.mot_joint_attention_backward_workspace_bytes(64, 4, 2, 64, 2)
    assert need >= 64 + 4 * 64 * 4 and need % 16 == 0
    assert back(wsb=need - 1) == MOT_ERR_WORKSPACE
    for bad in ((0, 4, 2, 64, 1), (64, 3, 2, 64, 1), (64, 4, 2, 96, 1), (64, 4, 2, 64, 0), ((1 << 24) + 1, 4, 2, 64, 1)):
        assert lib.mot_joint_attention_backward_workspace_bytes(*bad) == 0, bad


@pytest.mark.parametrize("name", ["mot_qk_norm_rope_backward", "mot_qk_norm_rope_backward_fp32"])
def test_qk_norm_rope_backward_rejects(lib, name):
    base = dict(d=A, x=B, qw=C, kw=C, pos=E, cs=F, P=64, T=64, Hq=4, Hkv=2, D=64, eps=1e-6, ws=G, wsb=1 << 20, dx=A, dw=H,
                sets=3, scratch=B, sb=1 << 30)

    def f(**kw):
        a = {**base, **kw}
        return getattr(lib, name)(a["d"], a["x"], a["qw"], a["kw"], a["pos"], a["cs"], a["P"], a["T"], a["Hq"], a["Hkv"],
                                  a["D"], a["eps"], a["ws"], a["wsb"], a["dx"], a["dw"], a["sets"], a["scratch"], a["sb"], None)

    for arg in ("d", "x", "qw", "kw", "pos", "cs", "ws", "dx", "scratch"):
        assert f(**{arg: None}) == MOT_ERR_NULL, arg
        assert f(**{arg: MIS}) == MOT_ERR_ALIGN, arg
    assert f(dw=MIS) == MOT_ERR_ALIGN
    for bad in (dict(T=0), dict(T=(1 << 24) + 1), dict(D=96), dict(Hq=0), dict(Hkv=0), dict(Hq=1025), dict(Hkv=1025)):
        assert f(**bad) == MOT_ERR_GEOMETRY, bad
    for bad in (dict(P=0), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(sets=0), dict(sets=4)):
        assert f(**bad) == MOT_ERR_ARG, bad
    assert f(wsb=100) == MOT_ERR_WORKSPACE
    need = lib.mot_qk_norm_rope_backward_workspace_bytes(64, 64)
    assert need > 0 and f(sb=need - 1) == MOT_ERR_WORKSPACE
    fine = (0, MOT_ERR_NULL, MOT_ERR_ALIGN, MOT_ERR_GEOMETRY, MOT_ERR_ARG, MOT_ERR_WORKSPACE)
    assert f() not in fine and f(dw=None, sets=0, scratch=None, sb=0) not in fine  # the device is what is left
    for bad in ((0, 64), ((1 << 24) + 1, 64), (64, 96)):
        assert lib.mot_qk_norm_rope_backward_workspace_bytes(*bad) == 0


def test_adamw_step_rejects(lib):
    base = dict(p=A, p16=B, g=C, m=E, v=F, scales=G, n=1000, weight_decay=0.1, flags=2)

    def f(count=1, hyper=H, ws=A, wsb=64, second=None, **kw):
        table = (mot._AdamWTensor * 2)(*(mot._AdamWTensor(**{**base, **kw}), mot._AdamWTensor(**{**base, **(second or {})})))
        return lib.mot_adamw_step(ctypes.addressof(table), count, hyper, 0, ws, wsb, None)

    for name in ("p", "g", "m", "v", "scales"):
        assert f(**{name: None}) == MOT_ERR_NULL, name
        assert f(count=2, second={name: None}) == MOT_ERR_NULL, name
        assert f(**{name: MIS + 4}) == MOT_ERR_ALIGN, name
    assert lib.mot_adamw_step(None, 1, H, 0, A, 64, None) == MOT_ERR_NULL
    assert f(hyper=None) == MOT_ERR_NULL and f(ws=None) == MOT_ERR_NULL
    assert f(hyper=MIS) == MOT_ERR_ALIGN and f(ws=MIS) == MOT_ERR_ALIGN and f(p16=MIS) == MOT_ERR_ALIGN
    assert f(p=MIS) == MOT_ERR_ALIGN and f(flags=0, scales=None, p=MIS) == MOT_ERR_ALIGN
    for bad in (dict(count=0), dict(count=-1), dict(count=65537), dict(n=0), dict(n=-5), dict(n=(1 << 40) + 1)):
        assert f(**bad) == MOT_ERR_GEOMETRY, bad
    for bad in (dict(flags=4), dict(flags=-1), dict(weight_decay=-0.1), dict(weight_decay=float("nan")),
                dict(weight_decay=float("inf"))):
        assert f(**bad) == MOT_ERR_ARG, bad
    assert f(wsb=63) == MOT_ERR_WORKSPACE
    fine = (0, MOT_ERR_NULL, MOT_ERR_ALIGN, MOT_ERR_GEOMETRY, MOT_ERR_ARG, MOT_ERR_WORKSPACE)
    assert f() not in fine and f(flags=0, scales=None, p16=None) not in fine and f(scales=MIS) not in fine


def test_binding_names_what_it_refuses():
    x, ok = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(4)
    with pytest.raises(TypeError, match="dout"):
        mot.mot_joint_attention_backward(None, x, x, x, x, 1, 1, 64, x)
    with pytest.raises(ValueError, match="qkv must be a CUDA tensor"):
        mot.mot_joint_attention_lse(x, x, 1, 1, 64, x)
    with pytest.raises(ValueError, match="d_out must be a CUDA tensor"):
        mot.mot_qk_norm_rope_backward(x, x, x, x, x, x, 1, 1, 64, 1e-6, x)
    with pytest.raises(TypeError, match="rope_cs_f32"):
        mot.mot_qk_norm_rope_backward_fp32(x, x, x, x, x, x, 1, 1, 64, 1e-6, x)
    with pytest.raises(ValueError, match="one entry"):
        mot.AdamWTensors([ok], [], [ok], [ok])
    with pytest.raises(ValueError, match="one entry"):
        mot.AdamWTensors([], [], [], [])
    with pytest.raises(ValueError, match=r"params\[0\] must be a CUDA tensor"):
        mot.AdamWTensors([ok], [ok], [ok], [ok])
    with pytest.raises(TypeError, match="AdamWTensors"):
        mot.mot_adamw_step([ok], ok, ok)
