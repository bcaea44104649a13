"""Buffers that a caller leaves to the binding belong to the stream that the call is launched on, whatever the current one is:
for every call that makes some, without a GPU on a stand-in for torch; on a GPU beside a stream that is busy."""

import contextlib

import pytest
import torch

import mixture_transformers_token_gb300 as mot
from mixture_transformers_token_gb300 import workloads as W

from _util import assert_bitwise, need_gpu

DEV = "cuda"
BF, F32, U8, I32, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64


# ---------------------------------------------------------------------------
# without a GPU
# ---------------------------------------------------------------------------

class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class FakeTensor:
    is_cuda, device = True, "a GPU"

    def __init__(self, shape, dtype, stream=None):
        self.shape, self.dtype, self.stream, self.recorded = tuple(shape), dtype, stream, []

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def data_ptr(self):
        return 4096

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


class FakeTorch:
    """torch as the binding uses it, its tensors noting the stream that they were made on."""

    def __init__(self):
        self.cuda, self.made, self.current, self.default = self, [], FakeStream(11), FakeStream(0)
        self.Stream, self.ExternalStream = FakeStream, lambda handle, device: FakeStream(handle)

    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, shape, dtype, device):
        assert device == "a GPU"
        self.made.append(FakeTensor(shape if isinstance(shape, tuple) else (shape,), dtype, self.current.cuda_stream))
        return self.made[-1]

    zeros = empty

    def empty_like(self, t):
        return self.empty(t.shape, t.dtype, t.device)

    zeros_like = empty_like

    def current_stream(self, device):
        return self.current

    def default_stream(self, device):
        return self.default

    @contextlib.contextmanager
    def stream(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before


def _t(dtype, *shape):
    return FakeTensor(shape, dtype)


T, H, HQ, HKV, D, N = 6, 256, 4, 2, 64, 512
ROWS, WS, POS, MOD = _t(BF, T, H), _t(U8, 4096), _t(I32, T), _t(U8, T)
QKV, OUT, SEQS, NORM, TABLE = _t(BF, T, N), _t(BF, T, HQ * D), _t(I32, 1, 5), _t(BF, 2, D), _t(BF, 9, D // 2, 2)
CACHE, LATENT, PLANE = _t(BF, 3, HKV, 16, D), _t(F32, 2, 300), _t(BF, 2, 300)

# each call and how many buffers it makes, how many of them it returns
CALLS = {
    "route_plan": (lambda s: mot.mot_route_plan(MOD, stream=s), 1, 1),
    "add_rmsnorm": (lambda s: mot.mot_fused_add_rmsnorm(ROWS, ROWS, _t(BF, 2, H), MOD, 1e-6, stream=s), 2, 2),
    "qkv": (lambda s: mot.mot_routed_qkv_norm_rope(ROWS, _t(BF, 2, N, H), NORM, NORM, POS, TABLE, HQ, HKV, D, 1e-6, WS, stream=s), 1, 1),
    "gemm": (lambda s: mot.mot_routed_gemm(ROWS, _t(BF, 2, N, H), WS, stream=s), 1, 1),
    "gemm_noalloc": (lambda s: mot.mot_routed_gemm_noalloc(ROWS, _t(BF, 2, N, H), MOD, stream=s), 1, 1),
    "gather_rows": (lambda s: mot.mot_gather_rows(ROWS, WS, stream=s), 1, 1),
    "interleave": (lambda s: mot.mot_swiglu_interleave(_t(BF, 2, N, H), _t(BF, 2, N, H), stream=s), 1, 1),
    "gemm_dx": (lambda s: mot.mot_routed_gemm_dx(QKV, _t(BF, 2, N, H), WS, stream=s), 1, 1),
    "gemm_dw": (lambda s: mot.mot_routed_gemm_dw(QKV, ROWS, WS, stream=s), 1, 1),
    "attention": (lambda s: mot.mot_joint_attention(QKV, SEQS, HQ, HKV, D, WS, stream=s), 1, 1),
    "attention_lse": (lambda s: mot.mot_joint_attention_lse(QKV, SEQS, HQ, HKV, D, WS, stream=s), 2, 2),
    "attention_backward": (lambda s: mot.mot_joint_attention_backward(OUT, QKV, OUT, _t(F32, HQ, T), SEQS, HQ, HKV, D, WS, stream=s), 1, 1),
    "qk_norm_rope_backward": (lambda s: mot.mot_qk_norm_rope_backward(QKV, QKV, NORM, NORM, POS, TABLE, HQ, HKV, D, 1e-6, WS, stream=s), 3, 2),
    "decode": (lambda s: mot.mot_paged_decode_attention(QKV, _t(I32, T, 2), POS, CACHE, CACHE, HQ, WS, stream=s), 1, 1),
    "rmsnorm_backward": (lambda s: mot.mot_add_rmsnorm_backward(ROWS, ROWS, _t(BF, 2, H), 1e-6, WS, stream=s), 2, 2),
    "rmsnorm_dweight": (lambda s: mot.mot_rmsnorm_dweight(_t(F32, 4, T, 64), WS, stream=s), 1, 1),
    "cfg": (lambda s: mot.mot_cfg_combine_renorm(PLANE, PLANE, PLANE, _t(F32, 2, 6), stream=s), 2, 1),
    "sde_step": (lambda s: mot.mot_flow_sde_step(LATENT, LATENT, LATENT, _t(F32, 2, 2), stream=s), 3, 2),
    "cfg_sde_step": (lambda s: mot.mot_flow_cfg_sde_step(PLANE, PLANE, None, _t(F32, 2, 6), LATENT, LATENT, _t(F32, 2, 2), stream=s), 3, 2),
    "noise": (lambda s: mot.mot_flow_noise(_t(I64, 2), 3, 300, stream=s), 1, 1),
}


class FakeLibrary:
    def __getattr__(self, name):
        return lambda *args: 640 if name.endswith("_bytes") else 0


@pytest.fixture
def fake(monkeypatch):
    f = FakeTorch()
    monkeypatch.setattr(mot, "torch", f)
    monkeypatch.setattr(mot, "_lib", FakeLibrary)
    monkeypatch.setattr(mot, "_dev", lambda t, *args: t.data_ptr())
    monkeypatch.setattr(mot, "_raw_stream", lambda device: f.current.cuda_stream)
    return f


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream,handle", [(FakeStream(5), 5), (5, 5), (0, 0), (FakeStream(11), 11), (None, 11)],
                         ids=["stream", "handle", "default", "current", "none"])
def test_buffers_are_made_on_the_launch_stream(fake, call, stream, handle):
    run, made, returned = CALLS[call]
    got = run(stream)
    got = [t for t in (got if isinstance(got, tuple) else (got,)) if t in fake.made]
    assert len(fake.made) == made and len(got) == returned
    assert [t.stream for t in fake.made] == [handle] * made
    # what is returned may be used on the current stream, what is the call's own is let go on the launch stream alone
    assert all(t.recorded == ([11] if handle != 11 else []) for t in got)
    assert not any(t.recorded for t in fake.made if t not in got)
    assert fake.current.cuda_stream == 11


# ---------------------------------------------------------------------------
# on a GPU
# ---------------------------------------------------------------------------

class Step:
    """Inputs of the calls whose buffers are filled before the launch or let go after it, and what the calls give."""

    def __init__(self):
        self.T, self.Hq, self.Hkv, self.D = 700, 4, 2, 128
        r = W.rng_for(3, 970)
        n = (self.Hq + 2 * self.Hkv) * self.D
        self.qkv, self.d = (W.bf16_normal(r, (self.T, n)).to(DEV) for _ in range(2))
        self.dout = W.bf16_normal(r, (self.T, self.Hq * self.D)).to(DEV)
        self.w = W.bf16_normal(r, (2, self.D), mean=1.0, std=0.1).to(DEV)
        self.seqs = torch.tensor([(0, 0, 650, 650, 300)], dtype=torch.int32, device=DEV)
        self.pos = torch.arange(self.T, dtype=torch.int32, device=DEV)
        self.cs = mot.mot_rope_table_fill_host(1e4, self.D, self.T).to(DEV)
        self.plan = mot.mot_route_plan((torch.arange(self.T, device=DEV) % 3 == 0).to(U8))
        size = mot.mot_joint_attention_backward_workspace_bytes(self.T, self.Hq, self.Hkv, self.D, 1)
        self.ws = torch.zeros(size, dtype=U8, device=DEV)

    def attention(self, stream=None):
        h = (self.Hq, self.Hkv, self.D)
        out, lse = mot.mot_joint_attention_lse(self.qkv, self.seqs, *h, self.ws, stream=stream)
        plain = mot.mot_joint_attention(self.qkv, self.seqs, *h, self.ws, stream=stream)
        return out, lse, plain, mot.mot_joint_attention_backward(self.dout, self.qkv, out, lse, self.seqs, *h, self.ws, stream=stream)

    def norm(self, stream=None, d=None):
        return mot.mot_qk_norm_rope_backward(self.d if d is None else d, self.qkv, self.w, self.w, self.pos, self.cs, self.Hq,
                                             self.Hkv, self.D, 1e-6, self.plan, stream=stream)


def _keep_busy(n=40):
    """Some 10 ms of work on the current stream."""
    a = torch.ones((8192, 8192), dtype=BF, device=DEV)
    b = torch.empty_like(a)
    for _ in range(n):
        torch.mm(a, a, out=b)
    return a, b


def _same(got, want):
    for a, b in zip(got, want):
        assert_bitwise(a.view(BF), b.view(BF), "on another stream")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_fills_beside_a_busy_current_stream(kind):
    need_gpu()
    s, side = Step(), torch.cuda.Stream()
    want = *s.attention(), *s.norm()
    torch.cuda.synchronize()
    stream = side if kind == "stream" else side.cuda_stream
    held = _keep_busy()
    got = *s.attention(stream), *s.norm(stream)
    torch.cuda.synchronize()
    _same(got, want)
    del held


@pytest.mark.gpu
def test_on_the_default_stream_from_another():
    need_gpu()
    s = Step()
    want = *s.attention(), *s.norm()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        held = _keep_busy()
        got = *s.attention(0), *s.norm(0)
    torch.cuda.synchronize()
    _same(got, want)
    del held


@pytest.mark.gpu
def test_memory_let_go_while_the_launch_stream_is_busy():
    # scratch is let go at the call's return, long before the kernels run: the current stream's next tensors have other memory
    need_gpu()
    s, side = Step(), torch.cuda.Stream()
    want = s.norm()
    size = mot.mot_qk_norm_rope_backward_workspace_bytes(s.T, s.D)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        held = _keep_busy()
    got = s.norm(side)
    mine = [torch.full((size,), 7, dtype=U8, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    _same(got, want)
    assert all(bool((t == 7).all()) for t in mine)
    del held


@pytest.mark.gpu
def test_results_let_go_while_the_current_stream_reads_them():
    # results of a call on another stream, read late by the current one and let go at once: the next call has other memory
    need_gpu()
    s, side = Step(), torch.cuda.Stream()
    more = s.d * 2
    want = [s.norm(d=d)[0] for d in (s.d, more)]
    torch.cuda.synchronize()
    got = s.norm(side)[0]
    torch.cuda.current_stream().wait_stream(side)
    held = _keep_busy()
    copy = got.clone()
    del got
    other = s.norm(side, more)[0]
    torch.cuda.synchronize()
    _same([copy, other], want)
    del held


@pytest.mark.gpu
def test_captured_on_a_stream_beside_the_capturing_one():
    need_gpu()
    s, side, graph = Step(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    want = *s.attention(), *s.norm()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        s.norm(side)  # results that nobody keeps
        got = *s.attention(side), *s.norm(side)
        main.wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(2):
        for t in (*got, *copies):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _same(got, want)
        _same(copies, want)
