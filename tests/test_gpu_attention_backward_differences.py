"""Joint attention's backward pass against differences of the 64-bit forward, along directions in which a wrong gradient shows: the
gradient's own, of the q, the k and the v columns each."""

import numpy as np
import pytest
import torch

from oracle import mot_oracle as O

from _util import f64, need_gpu
from test_gpu_attention_backward import _backward, _forward, _inputs

PACKS = {
    "prompt_and_latents": ([(0, 0, 90, 90, 60), (90, 0, 110, 150, 0)], 200),
    "shared_prompt": ([(0, 0, 137, 137, 137), (137, 0, 60, 137, 0), (197, 0, 5, 137, 0)], 210),
    "cached_prefix": ([(150, 0, 40, 190, 40)], 190),
}
HEADS = [(4, 2, 64), (7, 1, 128)]


def _parts(Hq, Hkv, D):
    return slice(0, Hq * D), slice(Hq * D, (Hq + Hkv) * D), slice((Hq + Hkv) * D, (Hq + 2 * Hkv) * D)


def _differences(d, x, w, out, lse, seqs, Hq, Hkv, D):
    """For each of the q, k and v columns, along the unit direction u of the 64-bit gradient there: the difference quotient of f(x) =
    sum w attention(x), the product of d with u, and a bound on their distance."""
    exact = O.g_joint_attention(x, seqs, Hq, Hkv, D)["out_pre"]
    l64, _ = O.g_attention_lse(x, seqs, Hq, Hkv, D)
    true = O.g_joint_attention_backward(w, x, exact, l64, seqs, Hq, Hkv, D)["dqkv"]
    g = O.g_joint_attention_backward(w, x, out, lse, seqs, Hq, Hkv, D)  # of the rounded out and lse that d was formed from
    rows = []
    for cols in _parts(Hq, Hkv, D):
        u = np.zeros_like(x)
        u[:, cols] = true[:, cols] / np.linalg.norm(true[:, cols])
        h = 1e-2  # for about 20000 values of unit size: 1e-4 of each
        f = [float((O.g_joint_attention(x + k * h * u, seqs, Hq, Hkv, D)["out_pre"] * w).sum()) for k in (1, -1, 2, -2)]
        near, far = (f[0] - f[1]) / (2 * h), (f[2] - f[3]) / (4 * h)
        # the kernel's own error, as counted; what the rounding of out and lse changes, as it is; the difference quotient's error, of
        # third derivatives: a third of the distance to the quotient of twice the step, with what is of fifth order counted as that again
        bound = float((g["err"] * np.abs(u)).sum()) + abs(float(((g["dqkv"] - true) * u).sum())) + abs(near - far) + 1e-9
        rows.append((near, float((d * u).sum()), bound))
    return rows


def _wrong(d, Hq, Hkv, D):
    """Gradients that the comparison has to refuse, and in which of the three columns."""
    q, k, v = _parts(Hq, Hkv, D)
    yield np.zeros_like(d), (0, 1, 2)
    yield -d, (0, 1, 2)
    for i, cols in enumerate((q, k, v)):
        for f in (0.0, 0.5, 2.0):
            x = d.copy()
            x[:, cols] *= f
            yield x, (i,)
    x = d.copy()
    x[:, k], x[:, v] = d[:, v], d[:, k]
    yield x, (1, 2)
    yield d[::-1], (0, 1, 2)


def _assert_close_and_sharp(d, x, w, out, lse, seqs, Hq, Hkv, D):
    for part, (want, got, bound) in zip("qkv", _differences(d, x, w, out, lse, seqs, Hq, Hkv, D)):
        assert abs(want - got) <= bound, (part, want, got, bound)
        assert bound <= 0.2 * abs(want), (part, want, bound)
    for bad, where in _wrong(d, Hq, Hkv, D):
        rows = _differences(bad, x, w, out, lse, seqs, Hq, Hkv, D)
        for i in where:
            want, got, bound = rows[i]
            assert abs(want - got) > bound, ("a wrong gradient passes", i, want, got, bound)


def test_the_comparison_on_the_oracle():
    # the oracle's gradient, rounded once, passes and wrong ones do not
    Hq, Hkv, D = HEADS[0]
    seqs, T = PACKS["prompt_and_latents"]
    rng = np.random.default_rng(7)
    x, w = O.bf16(rng.standard_normal((T, (Hq + 2 * Hkv) * D))), O.bf16(rng.standard_normal((T, Hq * D)))
    out = O.g_joint_attention(x, seqs, Hq, Hkv, D)["out"]
    lse = O.g_attention_lse(x, seqs, Hq, Hkv, D)[0].astype(np.float32).astype(np.float64)
    d = O.bf16(O.g_joint_attention_backward(w, x, out, lse, seqs, Hq, Hkv, D)["dqkv"])
    _assert_close_and_sharp(d, x, w, out, lse, seqs, Hq, Hkv, D)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("pack", PACKS)
def test_gradient_along_its_own_directions(pack, Hq, Hkv, D):
    need_gpu()
    seqs, T = PACKS[pack]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=T + Hq)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    d = torch.where(d == 7.0, torch.zeros_like(d), d)
    _assert_close_and_sharp(f64(d), f64(qkv), f64(dout), f64(out), lse.double().cpu().numpy(), seqs, Hq, Hkv, D)
