"""The paged key-value cache without a GPU: the oracle's quantiser against brute force, and the
entry points' refusals (made before any CUDA call)."""

import numpy as np
import pytest

import mixture_transformers_token_gb300 as mot
from mixture_transformers_token_gb300 import build as mot_build
from oracle import mot_oracle as O

MOT_ERR_NULL, MOT_ERR_ALIGN, MOT_ERR_GEOMETRY, MOT_ERR_WORKSPACE, MOT_ERR_ARG = 1, 2, 3, 5, 8
A, B, C, E, F = (n << 20 for n in (1, 2, 3, 5, 6))   # fake, aligned, not NULL
MIS = (4 << 20) + 8


@pytest.fixture(scope="module")
def lib():
    mot_build.build()
    return mot.load_library()


def test_e4m3_values_and_rounding_by_brute_force():
    v = O.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[126] == 448.0 and np.all(np.diff(v) > 0)
    rng = np.random.default_rng(1)
    x = np.concatenate([v, (v[1:] + v[:-1]) / 2, rng.uniform(0, 448, 500), 2.0 ** rng.uniform(-14, 8, 500)])
    x = np.concatenate([x, -x])
    got = O.e4m3_round(x)
    for a, g in zip(x, got):
        d = np.abs(v - abs(a))
        near = np.flatnonzero(d == d.min())
        code = near[0] if len(near) == 1 else near[near % 2 == 0][0]
        assert g == np.copysign(v[code], a)
    assert np.isnan(O.e4m3_round(np.nan))


def test_quantise_takes_the_smallest_scale_that_holds_the_vector():
    rng = np.random.default_rng(2)
    x = O.bf16(rng.standard_normal((400, 64)) * np.exp2(rng.integers(-100, 100, (400, 1))))
    x[0] = 0
    x[1] = 448.0 * 2.0 ** -70   # below the smallest scale's share of the range
    x[2, 3] = 448.0 * 2.0 ** 5
    x[2, 4:] = 0
    y, s = O.kv_quantise(x)
    a = np.abs(x).max(-1)
    e = np.log2(s)
    assert np.all(e == np.round(e)) and np.all(e >= -64) and np.all(a <= 448 * s)
    assert np.all((e == -64) | (a > 448 * s / 2)) and s[0] == s[1] == 2.0 ** -64
    # half a step of a normal value is 2^-4 of it; subnormals lose at most half of 2^-9 scale
    assert np.all(np.abs(y * s[:, None] - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s[:, None]))
    x[5, 9], x[6, 1] = np.inf, np.nan
    y, s = O.kv_quantise(x)
    assert np.isnan(s[5]) and np.isnan(s[6]) and np.isfinite(s[7])


def test_paged_decode_golden_is_joint_attention_of_the_last_row():
    rng = np.random.default_rng(3)
    Hq, Hkv, D, n = 6, 2, 8, 37
    qkv = rng.standard_normal((n, (Hq + 2 * Hkv) * D))
    g = O.g_joint_attention(qkv, [(0, 0, n, n, n)], Hq, Hkv, D)["out_pre"][-1]
    k = qkv[:, Hq * D:(Hq + Hkv) * D].reshape(n, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:].reshape(n, Hkv, D)
    got = O.g_paged_decode(qkv[-1:, :Hq * D].reshape(1, Hq, D), [k], [v], Hq, Hkv)
    np.testing.assert_allclose(got["out_pre"].reshape(-1), g, rtol=1e-12, atol=1e-14)
    assert np.all(got["p_abs_v"] >= np.abs(got["out_pre"]) - 1e-12)
    empty = O.g_paged_decode(qkv[-1:, :Hq * D].reshape(1, Hq, D), [k[:0]], [v[:0]], Hq, Hkv)
    assert not empty["out_pre"].any()


def _cache_calls(lib):
    """Both directions as call(**changes) of a valid argument list."""
    base = dict(qkv=A, T=64, Hq=4, Hkv=2, D=64, slots=B, kt=1, n=10, page=16, k=C, v=E, sc=F, ws=A, wsb=64)

    def write(**kw):
        a = {**base, **kw}
        return lib.mot_kv_cache_write(a["qkv"], a["T"], a["Hq"], a["Hkv"], a["D"], a["slots"], a["kt"], a["n"],
                                      a["page"], a["k"], a["v"], a["sc"], a["ws"], a["wsb"], None)

    def read(**kw):
        a = {**base, **kw}
        return lib.mot_kv_cache_read(a["k"], a["v"], a["sc"], a["kt"], a["n"], a["page"], a["slots"], a["T"], a["Hq"],
                                     a["Hkv"], a["D"], a["qkv"], a["ws"], a["wsb"], None)

    def decode(**kw):
        a = {**base, "wsb": 1 << 30, "scale": 0.125, "table": B, "lens": C, "mp": 10, "out": E, **kw}
        return lib.mot_paged_decode_attention(a["qkv"], a["T"], a["Hq"], a["Hkv"], a["D"], a["table"], a["lens"],
                                              a["mp"], a["kt"], a["n"], a["page"], a["k"], a["v"], a["sc"],
                                              a["scale"], a["ws"], a["wsb"], a["out"], None)

    return write, read, decode


def test_cache_calls_reject(lib):
    for f in _cache_calls(lib):
        for name in ("qkv", "k", "v", "ws", "sc"):
            assert f(**{name: None}) == MOT_ERR_NULL, name
            assert f(**{name: MIS}) == MOT_ERR_ALIGN, name
        assert f(kt=2) == MOT_ERR_ARG and f(kt=-1) == MOT_ERR_ARG
        for bad in (dict(D=96), dict(D=256), dict(Hq=3), dict(Hkv=0), dict(Hq=0), dict(Hq=1025, Hkv=1), dict(page=8),
                    dict(page=24), dict(page=1040), dict(page=0), dict(n=0), dict(n=-1), dict(T=0),
                    dict(T=(1 << 24) + 1), dict(n=1 << 26), dict(n=1 << 62)):
            assert f(**bad) == MOT_ERR_GEOMETRY, bad
        assert f(wsb=63) == MOT_ERR_WORKSPACE
        # a bf16 cache has no scales; what is left to fail is the device
        assert f(kt=0, sc=None) not in (0, MOT_ERR_NULL, MOT_ERR_ALIGN, MOT_ERR_GEOMETRY, MOT_ERR_ARG)


def test_decode_rejects(lib):
    write, read, f = _cache_calls(lib)
    for name in ("table", "lens", "out"):
        assert f(**{name: None}) == MOT_ERR_NULL, name
        assert f(**{name: MIS + 2}) == MOT_ERR_ALIGN, name
    assert f(out=MIS) == MOT_ERR_ALIGN
    for call in (write, read):
        assert call(slots=None) == MOT_ERR_NULL and call(slots=MIS + 2) == MOT_ERR_ALIGN
        assert call(slots=MIS + 4) not in (0, MOT_ERR_ALIGN)     # an int32 array may start anywhere
    assert f(table=MIS + 4, lens=MIS) not in (0, MOT_ERR_ALIGN)
    assert f(mp=0) == MOT_ERR_GEOMETRY
    assert f(mp=(1 << 26) + 1) == MOT_ERR_GEOMETRY
    assert f(mp=(1 << 20) + 1) == MOT_ERR_GEOMETRY            # more than 2^24 keys a row
    assert f(mp=1 << 20, T=1) not in (0, MOT_ERR_GEOMETRY)
    assert f(T=1 << 22, Hq=1024, Hkv=1024) == MOT_ERR_GEOMETRY  # R * Hq
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert f(scale=scale) == MOT_ERR_ARG


def test_decode_workspace_bytes(lib):
    f = lib.mot_paged_decode_workspace_bytes
    assert f(1, 4, 2, 64, 1, 16) >= 64
    for bad in ((0, 4, 2, 64, 1, 16), (1, 3, 2, 64, 1, 16), (1, 4, 2, 96, 1, 16), (1, 4, 2, 64, 0, 16),
                (1, 4, 2, 64, 1, 8), (1, 4, 2, 64, (1 << 26) + 1, 16), ((1 << 24) + 1, 4, 2, 64, 1, 16)):
        assert f(*bad) == 0, bad
    for args in ((1, 28, 4, 128, 8192, 16), (64, 28, 4, 128, 512, 16), (3, 16, 1, 64, 100, 48)):
        n = f(*args)
        need = n - 1
        write, read, decode = _cache_calls(lib)
        R, Hq, Hkv, D, mp, page = args
        assert n % 16 == 0
        assert decode(T=R, Hq=Hq, Hkv=Hkv, D=D, mp=mp, page=page, wsb=need) == MOT_ERR_WORKSPACE
