"""Joint attention's backward pass over query ranges that overlap: no work where they have more than T rows in all."""

import pytest
import torch

import mixture_transformers_token_gb300 as mot

from _util import assert_bitwise, need_gpu
from test_gpu_attention_backward import _backward, _forward, _inputs, _ws

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("n", [2, 64, 65, 3000])
@pytest.mark.parametrize("causal", [0, 200])
def test_more_query_rows_than_there_are(n, causal):
    Hq, Hkv, D, T = 4, 2, 64, 200
    good = [(0, 0, T, T, causal)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=31)
    s, out, lse = _forward(qkv, good, Hq, Hkv, D)
    want = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    many = torch.tensor(good * n, dtype=torch.int32, device=DEV)
    d = _backward(dout, qkv, out, lse, many, Hq, Hkv, D, flags=mot.DEV_BAD_SEQUENCE)
    assert bool((d == 7.0).all())
    # the workspace serves the next call
    ws, d = _ws(T, Hq, Hkv, D, n), torch.full_like(qkv, 7.0)
    mot.mot_joint_attention_backward(dout, qkv, out, lse, many, Hq, Hkv, D, ws, dqkv=d)
    assert mot.mot_device_status(ws) == mot.DEV_BAD_SEQUENCE
    ws[:64] = 0
    assert_bitwise(mot.mot_joint_attention_backward(dout, qkv, out, lse, s, Hq, Hkv, D, ws, dqkv=d), want, "the next call")
    assert mot.mot_device_status(ws) == 0


def test_as_many_query_rows_as_there_are():
    # every row is a query, and one descriptor is bad: the others' work is done
    Hq, Hkv, D, T = 4, 2, 64, 200
    good = [(0, 0, 120, 120, 50), (120, 120, 80, 80, 80)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=32)
    s, out, lse = _forward(qkv, good, Hq, Hkv, D)
    want = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    for n in (1, 70):
        seqs = torch.tensor(good + [(0, 0, T, 0, 0)] * n, dtype=torch.int32, device=DEV)
        assert_bitwise(_backward(dout, qkv, out, lse, seqs, Hq, Hkv, D, flags=mot.DEV_BAD_SEQUENCE), want, f"{n} bad ones")
