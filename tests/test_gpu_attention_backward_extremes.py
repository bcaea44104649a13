"""Joint attention's backward pass at the ends of its geometry: the most heads, more descriptors than rows."""

import pytest

from _util import assert_bitwise, need_gpu
from test_gpu_attention_backward import _backward, _check, _forward, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("Hq,Hkv,D,T", [(1024, 1, 64, 140), (1024, 1, 128, 3), (1024, 1024, 64, 5), (1024, 2, 64, 40), (96, 32, 128, 20)])
def test_many_heads(Hq, Hkv, D, T):
    seqs = [(0, 0, T - 1, T - 1, T // 2), (T - 1, 0, 1, T, 1)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=Hq + T)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D)
    assert_bitwise(d, _backward(dout, qkv, out, lse, s, Hq, Hkv, D), "again")


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33])
@pytest.mark.parametrize("n", [63, 66, 5000])
def test_more_descriptors_than_rows(T, n):
    # keys alone, over every part of the rows, beside the one sequence that has queries
    Hq, Hkv, D = 4, 2, 64
    seqs = [(0, i % T, 0, 1 + i % (T - i % T), 0) for i in range(n)]
    seqs[n // 2] = (0, 0, T, T, T // 2)
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=T + n)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D)
    s, out, lse = _forward(qkv, [seqs[n // 2]], Hq, Hkv, D)
    alone = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    assert_bitwise(d[:, :Hq * D], alone[:, :Hq * D], "dq")
