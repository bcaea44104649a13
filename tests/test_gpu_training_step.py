"""A training step of one attention layer on the GPU, through the C ABI: the projection, attention with its softmax sums,
the output projection, back through all of them, and AdamW on the weights that the calls read. Every gradient is held
against a chain of the 64-bit formulas from the last layer's gradient on, within a bound that is carried through the
chain; the updated weights, against the emulator bit for bit; a captured step, against the same steps one by one."""

import numpy as np
import pytest
import torch

import mixture_transformers_token_gb300 as mot
from mixture_transformers_token_gb300 import workloads as W
from oracle import mot_oracle as O

from _util import assert_bitwise, f64, gemm_acc_err, need_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS, THETA = 1e-6, 1e6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Layer:
    """One layer's weights, their masters and states, and buffers of a step that a graph may hold."""

    def __init__(self, T, H, Hq, Hkv, D, seqs, seed, state="fp32", profile="bf16"):
        self.heads, self.N, self.seqs, self.T = (Hq, Hkv, D), (Hq + 2 * Hkv) * D, seqs, T
        r = W.rng_for(seed, 950)
        # latents (gen) are the rows that see a whole sequence, the prompt's rows are und
        mod = np.zeros(T, np.uint8)
        for q0, _, nq, _, nc in seqs:
            mod[q0 + nc:q0 + nq] = 1
        self.mod = torch.from_numpy(mod).to(DEV)
        self.pos = torch.from_numpy(r.integers(0, 4 * T, T).astype(np.int32)).to(DEV)
        self.s = torch.tensor(seqs, dtype=torch.int32, device=DEV)
        fill = mot.mot_rope_table_fill_host if profile == "bf16" else mot.mot_rope_table_fill_host_fp32
        self.cs = fill(THETA, D, 4 * T).to(DEV)
        self.forward_of_profile = mot.mot_routed_qkv_norm_rope if profile == "bf16" else mot.mot_routed_qkv_norm_rope_fp32
        self.x = W.bf16_normal(r, (T, H)).to(DEV)
        self.do = W.bf16_normal(r, (T, H)).to(DEV)
        self.w = {"qkv": W.bf16_normal(r, (2, self.N, H), std=H ** -0.5), "o": W.bf16_normal(r, (2, H, Hq * D), std=(Hq * D) ** -0.5),
                  "qn": W.bf16_normal(r, (2, D), mean=1.0, std=0.1), "kn": W.bf16_normal(r, (2, D), mean=1.0, std=0.1)}
        self.w = {k: v.to(DEV) for k, v in self.w.items()}
        self.g = {"qkv": torch.zeros((self.N, H), device=DEV), "o": torch.zeros((H, Hq * D), device=DEV)}
        self.dw = torch.full((2, 2, D), 7.0, device=DEV)  # of the norms; the und set's rows stay as they are
        grads = [self.g["qkv"], self.g["o"], self.dw[0, 1], self.dw[1, 1]]
        self.trained = [self.w["qkv"][1], self.w["o"][1], self.w["qn"][1], self.w["kn"][1]]
        self.master = [w.float() for w in self.trained]
        n = [w.numel() for w in self.trained]
        if state == "fp32":
            self.m, self.v = ([torch.zeros(i, device=DEV) for i in n] for _ in range(2))
            self.scales = None
        else:
            self.m, self.v = ([torch.zeros(i, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for i in n] for _ in range(2))
            self.scales = [torch.zeros((-(-i // 256), 2), device=DEV) for i in n]
        self.grads = grads
        self.adam = mot.AdamWTensors(self.master, grads, self.m, self.v, p16=self.trained, scales=self.scales,
                                     weight_decay=[0.1, 0.1, 0.0, 0.0])
        self.hyper = torch.zeros(16, device=DEV)
        self.ws = torch.zeros(mot.mot_workspace_bytes(T), dtype=torch.uint8, device=DEV)
        self.att_ws = torch.zeros(mot.mot_joint_attention_backward_workspace_bytes(T, Hq, Hkv, D, len(seqs)), dtype=torch.uint8,
                                  device=DEV)
        self.scratch = torch.empty(mot.mot_qk_norm_rope_backward_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
        self.opt_ws = torch.zeros(64, dtype=torch.uint8, device=DEV)

    def step(self, update=True):
        Hq, Hkv, D = self.heads
        w, ws, b = self.w, self.ws, {}
        mot.mot_route_plan(self.mod, ws=ws)
        b["proj"] = mot.mot_routed_gemm(self.x, w["qkv"], ws)
        b["qkv"] = self.forward_of_profile(self.x, w["qkv"], w["qn"], w["kn"], self.pos, self.cs, Hq, Hkv, D, EPS, ws)
        b["att"], b["lse"] = mot.mot_joint_attention_lse(b["qkv"], self.s, Hq, Hkv, D, self.att_ws)
        b["out"] = mot.mot_routed_gemm(b["att"], w["o"], ws)
        b["datt"] = mot.mot_routed_gemm_dx(self.do, w["o"], ws)
        mot.mot_routed_gemm_dw(self.do, b["att"], ws, expert=1, out=self.g["o"])
        b["dqkv"] = mot.mot_joint_attention_backward(b["datt"], b["qkv"], b["att"], b["lse"], self.s, Hq, Hkv, D, self.att_ws)
        b["dproj"], _ = mot.mot_qk_norm_rope_backward(b["dqkv"], b["proj"], w["qn"], w["kn"], self.pos, self.cs, Hq, Hkv, D, EPS,
                                                      ws, dw=self.dw, sets=mot.SET_GEN, scratch=self.scratch)
        b["dx"] = mot.mot_routed_gemm_dx(b["dproj"], w["qkv"], ws)
        mot.mot_routed_gemm_dw(b["dproj"], self.x, ws, expert=1, out=self.g["qkv"])
        if update:
            mot.mot_adamw_step(self.adam, self.hyper, self.opt_ws, seed=77)
        return b

    def status(self):
        return [mot.mot_device_status(x) for x in (self.ws, self.att_ws, self.opt_ws)]


def _routed_abs(a, w, mod):
    """|a| times |w| of each row's weight set, [T][K] by [2][K][N]."""
    return np.stack([np.abs(a[t]) @ np.abs(w[mod[t]]) for t in range(a.shape[0])])


def _attention_abs(e, qkv, out, lse, seqs, Hq, Hkv, D):
    """What a change of at most e of dout can change in dqkv."""
    d, sc = np.zeros_like(qkv), D ** -0.5
    for q0, k0, nq, nk, nc in seqs:
        see = O.attention_sees(nq, nk, nc)
        R, C = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            cq, ck, cv = (slice(i * D, (i + 1) * D) for i in (h, Hq + g, Hq + Hkv + g))
            q, k, v, eo = qkv[R, cq], qkv[C, ck], qkv[C, cv], e[R, cq]
            p = np.where(see, np.exp(np.where(see, q @ k.T * sc - lse[h, R][:, None], 0.0)), 0.0)
            ds = p * (eo @ np.abs(v).T + (eo * np.abs(out[R, cq])).sum(1)[:, None])
            d[R, cq] += sc * ds @ np.abs(k)
            d[C, ck] += sc * ds.T @ np.abs(q)
            d[C, cv] += p.T @ eo
    return d


def _norm_rope_abs(e, x, qn, kn, cos, sin, mod, Hq, Hkv, D):
    """What a change of at most e of d_out can change in dx and in dw [2][2][D]."""
    n, h2, T = Hq + Hkv, D // 2, x.shape[0]
    xx, ee = x[:, :n * D].reshape(T, n, D), e[:, :n * D].reshape(T, n, D)
    c, s = np.abs(cos)[:, None], np.abs(sin)[:, None]
    du = np.concatenate([ee[..., :h2] * c + ee[..., h2:] * s, ee[..., h2:] * c + ee[..., :h2] * s], -1)
    w = np.abs(np.concatenate([np.repeat(qn[mod][:, None], Hq, 1), np.repeat(kn[mod][:, None], Hkv, 1)], 1))
    rstd = 1.0 / np.sqrt((xx * xx).mean(-1, keepdims=True) + EPS)
    xh = np.abs(xx * rstd)
    dx = e.copy()
    dx[:, :n * D] = (rstd * (du * w + xh * (du * w * xh).mean(-1, keepdims=True))).reshape(T, -1)
    dw = np.stack([np.stack([(du * xh)[mod == i][:, hs].sum((0, 1)) for i in (0, 1)]) for hs in (slice(0, Hq), slice(Hq, n))])
    return dx, dw


SHAPES = {
    "prompt_and_latents": (130, 256, 4, 2, 64, [(0, 0, 90, 90, 60), (90, 90, 40, 40, 40)]),
    "shared_prompt": (300, 256, 6, 1, 128, [(0, 0, 141, 141, 141), (141, 0, 90, 141, 0), (231, 0, 69, 141, 0)]),
}


@pytest.mark.parametrize("profile", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients_through_the_layer(shape, profile):
    T, H, Hq, Hkv, D, seqs = SHAPES[shape]
    L = Layer(T, H, Hq, Hkv, D, seqs, seed=1, profile=profile)
    b = L.step(update=False)
    assert L.status() == [0, 0, 0]
    mod, h = L.mod.cpu().numpy(), {k: f64(v) for k, v in b.items() if k != "lse"}
    lse, w, x, do = b["lse"].double().cpu().numpy(), {k: f64(v) for k, v in L.w.items()}, f64(L.x), f64(L.do)
    half = O.U16

    def cast(v, e):  # a value within e, and its rounding to bf16
        return e + (np.abs(v) + e) * half

    # d att: the GEMM over H, one cast
    want = O.g_routed_gemm_dx(do, w["o"], mod)["dx_pre"]
    err = cast(want, gemm_acc_err(H, _routed_abs(do, w["o"], mod)))
    assert np.all(np.abs(h["datt"] - want) <= err)
    # dqkv: its own error at the gradient that it was given, and that gradient's error
    own = O.g_joint_attention_backward(h["datt"], h["qkv"], h["att"], lse, seqs, Hq, Hkv, D)
    assert np.all(np.abs(h["dqkv"] - own["dqkv"]) <= own["err"] + 1e-38) and own["written"].any(1).all()
    err = own["err"] + _attention_abs(err, h["qkv"], h["att"], lse, seqs, Hq, Hkv, D)
    want = O.g_joint_attention_backward(want, h["qkv"], h["att"], lse, seqs, Hq, Hkv, D)["dqkv"]
    assert np.all(np.abs(h["dqkv"] - want) <= err + 1e-38)
    # the projection's rows and the norms' weights
    cs = f64(L.cs)[L.pos.cpu().numpy()]
    args = (h["proj"], w["qn"], w["kn"], cs[..., 0], cs[..., 1], mod, Hq, Hkv, D)
    own = O.g_qk_norm_rope_backward(h["dqkv"], *args, EPS)
    assert np.all(np.abs(h["dproj"] - own["dx"]) <= own["err_dx"] + 1e-38)
    e_dx, e_dw = _norm_rope_abs(err, *args)
    g = O.g_qk_norm_rope_backward(want, *args, EPS)
    dw = L.dw.double().cpu().numpy()
    assert np.all(np.abs(dw - g["dw"])[:, 1] <= (own["err_dw"] + e_dw)[:, 1]) and np.all(dw[:, 0] == 7.0)
    want, err = g["dx"], own["err_dx"] + e_dx
    assert np.all(np.abs(h["dproj"] - want) <= err + 1e-38)
    # dx of the layer, and the gen set's weight gradients
    wx = O.g_routed_gemm_dx(want, w["qkv"], mod)["dx_pre"]
    acc = gemm_acc_err(L.N, _routed_abs(h["dproj"], w["qkv"], mod))
    assert np.all(np.abs(h["dx"] - wx) <= cast(wx, acc + _routed_abs(err, w["qkv"], mod)))
    gen = mod == 1
    for name, d, e, a in (("qkv", want, err, x), ("o", do, np.zeros_like(do), h["att"])):
        acc = gemm_acc_err(int(gen.sum()), (np.abs(d) + e)[gen].T @ np.abs(a)[gen])
        bound = acc + e[gen].T @ np.abs(a)[gen]
        assert np.all(np.abs(f64(L.g[name]) - O.g_routed_gemm_dw(d, a, mod, 1)) <= bound + 1e-38), name


@pytest.mark.parametrize("state", ["fp32", "e4m3"])
def test_steps_one_by_one_and_captured(state):
    T, H, Hq, Hkv, D, seqs = SHAPES["prompt_and_latents"]
    hyper = [mot.mot_adamw_hyper_host(1e-2, 0.9, 0.95, 1e-8, i + 1).to(DEV) for i in range(3)]
    one, graphed = (Layer(T, H, Hq, Hkv, D, seqs, seed=2, state=state) for _ in range(2))
    start = {k: v.clone() for k, v in one.w.items()}
    # one by one, each update against the emulator from the gradients that the step formed
    for i, row in enumerate(hyper):
        before = [[t.float().cpu().numpy() for t in x] for x in (one.master, one.m, one.v)]
        scales = [s.cpu().numpy() for s in one.scales] if one.scales else [None] * 4
        one.hyper.copy_(row)
        one.step()
        for j in range(4):
            want = O.e_adamw(before[0][j].reshape(-1), one.grads[j].cpu().numpy().reshape(-1), before[1][j], before[2][j],
                             row.cpu().numpy()[:9], [0.1, 0.1, 0.0, 0.0][j], j, i + 1, 77, scales[j])
            got = [one.master[j].cpu().numpy().reshape(-1), one.m[j].float().cpu().numpy(), one.v[j].float().cpu().numpy()]
            for a, e in zip(got, want):
                assert np.array_equal(a, np.asarray(e, np.float32)), (i, j)
            assert_bitwise(one.trained[j], one.master[j].to(torch.bfloat16), "the weights that the calls read")
    assert one.status() == [0, 0, 0]
    for k, v in one.w.items():
        assert_bitwise(v[0], start[k][0], "frozen " + k)
        assert not torch.equal(v[1], start[k][1]), k
    # captured once, replayed with each step's numbers
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        b = graphed.step()
    for row in hyper:
        graphed.hyper.copy_(row)
        graph.replay()
    torch.cuda.synchronize()
    assert graphed.status() == [0, 0, 0]
    for k in one.w:
        assert_bitwise(graphed.w[k], one.w[k], k)
    for x, y in zip(one.master + one.m + one.v + [one.dw], graphed.master + graphed.m + graphed.v + [graphed.dw]):
        assert torch.equal(x.float(), y.float())
    assert b["dx"].abs().sum() > 0
