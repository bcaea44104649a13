"""Joint attention's softmax sums and backward pass on the GPU, through the C ABI, against the fp64 oracle within the bound
that the oracle counts (roundings of the fp32 arithmetic, one bf16 rounding of P and dS, one of the result)."""

import numpy as np
import pytest
import torch

import mixture_transformers_token_gb300 as mot
from mixture_transformers_token_gb300 import workloads as W
from oracle import mot_oracle as O

from _util import assert_bitwise, bits, f64, need_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _ws(T, Hq, Hkv, D, n_seq):
    n = mot.mot_joint_attention_backward_workspace_bytes(T, Hq, Hkv, D, n_seq)
    ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV)  # whatever an allocator hands out
    ws[:64] = 0
    return ws


def _inputs(T, Hq, Hkv, D, seed, std=1.0):
    r = W.rng_for(seed, 700)
    return W.bf16_normal(r, (T, (Hq + 2 * Hkv) * D), std=std).to(DEV), W.bf16_normal(r, (T, Hq * D)).to(DEV)


def _forward(qkv, seqs, Hq, Hkv, D, scale=None):
    ws = torch.zeros(64, dtype=torch.uint8, device=DEV)
    s = torch.tensor(seqs, dtype=torch.int32, device=DEV).reshape(-1, 5)
    out, lse = mot.mot_joint_attention_lse(qkv, s, Hq, Hkv, D, ws, scale=scale)
    assert mot.mot_device_status(ws) == 0
    return s, out, lse


def _backward(dout, qkv, out, lse, s, Hq, Hkv, D, scale=None, flags=0):
    ws = _ws(qkv.shape[0], Hq, Hkv, D, s.shape[0])
    fill = torch.full_like(qkv, 7.0)
    d = mot.mot_joint_attention_backward(dout, qkv, out, lse, s, Hq, Hkv, D, ws, scale=scale, dqkv=fill)
    assert d is fill and mot.mot_device_status(ws) == flags
    return d


def _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D, scale=None):
    g = O.g_joint_attention_backward(f64(dout), f64(qkv), f64(out), lse.double().cpu().numpy(), seqs, Hq, Hkv, D, scale)
    got, w = f64(d), g["written"]
    assert np.all(got[~w] == 7.0), "columns that are nobody's were written"
    off = np.abs(got - g["dqkv"])
    bad = w & ~(off <= g["err"] + 1e-38)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), got[bad][:5], g["dqkv"][bad][:5], g["err"][bad][:5])
    return g


PACKS = {
    "one_row": ([(0, 0, 1, 1, 1)], 1),
    "one_latent_row": ([(2, 2, 1, 1, 0)], 4),
    "two": ([(0, 0, 2, 2, 2)], 2),
    "127": ([(0, 0, 127, 127, 127)], 127),
    "128": ([(0, 0, 128, 128, 128)], 128),
    "129": ([(0, 0, 129, 129, 100)], 130),
    "257_latents": ([(0, 0, 257, 257, 0)], 257),
    "300_and_213_unaligned": ([(3, 3, 300, 300, 200), (303, 303, 213, 213, 77)], 530),
    "many_short": ([(5 * i, 5 * i, 5, 5, i % 6) for i in range(40)], 203),
    "one_token_each": ([(i, i, 1, 1, i % 2) for i in range(150)], 150),
    # new rows after a cached prefix whose own queries are not here
    "cached_prefix": ([(250, 0, 70, 320, 70)], 320),
    "cached_prefix_one_new_token": ([(389, 0, 1, 390, 1)], 390),
    # a prompt, and three groups of latents that see its keys alone
    "shared_prompt": ([(0, 0, 137, 137, 137), (137, 0, 200, 137, 0), (337, 0, 64, 137, 0), (401, 0, 5, 137, 0)], 420),
    # keys of two sequences that overlap in part, queries that are not the last keys
    "overlapping_keys": ([(0, 100, 90, 200, 50), (90, 200, 140, 230, 0)], 440),
    "keys_without_queries": ([(0, 0, 0, 150, 0), (150, 140, 33, 60, 33)], 200),
    "nobody": ([(0, 0, 0, 1, 0)], 9),
}


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 7, 1), (128, 2, 2)])
@pytest.mark.parametrize("pack", PACKS)
def test_gradient_within_the_counted_bound(pack, D, Hq, Hkv):
    seqs, T = PACKS[pack]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=T + D)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D)
    assert_bitwise(d, _backward(dout, qkv, out, lse, s, Hq, Hkv, D), "the same call again")


@pytest.mark.parametrize("Hq,Hkv,D", [(28, 4, 128), (8, 8, 64), (12, 1, 64), (33, 3, 128), (16, 2, 128), (20, 4, 64)])
def test_head_groups(Hq, Hkv, D):
    seqs, T = [(1, 1, 150, 150, 90), (151, 151, 61, 61, 61)], 213
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=Hq)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 7, 1)])
def test_forward_lse(D, Hq, Hkv):
    for seqs, T in PACKS.values():
        qkv, _ = _inputs(T, Hq, Hkv, D, seed=T)
        s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
        ws = torch.zeros(64, dtype=torch.uint8, device=DEV)
        assert_bitwise(out, mot.mot_joint_attention(qkv, s, Hq, Hkv, D, ws), "out beside lse")
        want, s_abs = O.g_attention_lse(f64(qkv), seqs, Hq, Hkv, D)
        # the score's sum, then the sum of the weights: each is off by its argument's error (scores and their roundings),
        # two units of 2^x and the additions' (128 keys a block, then blocks); logf one unit
        n = max(x[3] for x in seqs)
        bound = s_abs * 2 * D * O.U32 + (np.abs(want) + s_abs) * 8 * O.U32 + (n + 40) * O.U32
        assert np.all(np.abs(lse.double().cpu().numpy() - want) <= bound)


def test_gradient_against_differences():
    # the whole chain forward and backward: f = sum dout out along random directions of the input
    Hq, Hkv, D, T = 4, 2, 64, 200
    seqs = [(0, 0, 90, 90, 60), (90, 0, 110, 150, 0)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=5)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    d[d == 7.0] = 0
    rng = np.random.default_rng(5)
    x, w = f64(qkv), f64(dout)
    g = O.g_joint_attention_backward(w, x, f64(out), lse.double().cpu().numpy(), seqs, Hq, Hkv, D)
    for _ in range(4):
        u = rng.standard_normal(x.shape)
        f = [float((O.g_joint_attention(x + k * 1e-4 * u, seqs, Hq, Hkv, D)["out_pre"] * w).sum()) for k in (1, -1)]
        # the kernel's gradient: its counted bound; the difference's own error: third derivatives, 1e-8 of u^3
        bound = float((g["err"] * np.abs(u)).sum()) + 1e-4 * float(np.linalg.norm(f64(d)))
        assert abs((f[0] - f[1]) / 2e-4 - float((f64(d) * u).sum())) <= bound


@pytest.mark.parametrize("scale", [0.02, 1.0, 3.0])
def test_scales_and_loud_scores(scale):
    # from nearly equal weights to rows whose weights are one key's alone
    Hq, Hkv, D, T = 4, 1, 64, 150
    seqs = [(0, 0, T, T, 100)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=9, std=2.0 if scale > 0.1 else 1.0)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D, scale)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D, scale)
    _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D, scale)


@pytest.mark.parametrize("scale", [2.0 ** -99, 2.0 ** 98])
def test_ends_of_the_scale_range(scale):
    # q and k shrink or grow against the scale, so that the scores are of unit size
    Hq, Hkv, D, T = 2, 1, 64, 140
    seqs = [(0, 0, T, T, 70)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=10)
    f = (0.125 / scale) ** 0.5
    f = 2.0 ** round(np.log2(f))
    qkv[:, :(Hq + Hkv) * D] *= f
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D, scale)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D, scale)
    _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D, scale)


def test_bits_do_not_depend_on_the_pack():
    Hq, Hkv, D, n = 7, 1, 128, 300
    qkv, dout = _inputs(n, Hq, Hkv, D, seed=11)
    s, out, lse = _forward(qkv, [(0, 0, n, n, 200)], Hq, Hkv, D)
    alone = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    for shift, others in ((77, [(0, 0, 77, 77, 40), (377, 377, 50, 50, 0)]), (128, [(0, 0, 128, 128, 0)]),
                          (1, []), (129, [(i, i, 1, 1, 1) for i in range(129)])):
        T = shift + n + 60
        big, bd = _inputs(T, Hq, Hkv, D, seed=shift)
        big[shift:shift + n], bd[shift:shift + n] = qkv, dout
        for at in (0, len(others)):
            seqs = others[:at] + [(shift, shift, n, n, 200)] + others[at:]
            s, out, lse = _forward(big, seqs, Hq, Hkv, D)
            d = _backward(bd, big, out, lse, s, Hq, Hkv, D)
            assert_bitwise(d[shift:shift + n], alone, f"shift {shift}")


def test_other_sequences_rows_may_hold_anything():
    Hq, Hkv, D = 4, 2, 64
    for T, seqs, mine in ((400, [(50, 50, 100, 100, 60), (150, 150, 90, 90, 90)], 0),
                          (300, [(0, 0, 130, 130, 130)], 0), (300, [(160, 100, 20, 70, 20)], 0)):
        qkv, dout = _inputs(T, Hq, Hkv, D, seed=T)
        s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
        clean = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
        q0, k0, nq, nk, _ = seqs[mine]
        own_q = torch.zeros(T, dtype=torch.bool, device=DEV)
        own_q[q0:q0 + nq] = True
        own_k = torch.zeros(T, dtype=torch.bool, device=DEV)
        own_k[k0:k0 + nk] = True
        for poison in (float("nan"), float("inf"), -3e38):
            x, do, o, l = qkv.clone(), dout.clone(), out.clone(), lse.clone()
            x[:, :Hq * D][~own_q] = poison
            x[:, Hq * D:][~own_k] = poison
            do[~own_q] = poison
            o[~own_q] = poison
            l[:, ~own_q] = poison
            d = _backward(do, x, o, l, s, Hq, Hkv, D)
            assert_bitwise(d[q0:q0 + nq, :Hq * D], clean[q0:q0 + nq, :Hq * D], "dq")
            assert_bitwise(d[k0:k0 + nk, Hq * D:], clean[k0:k0 + nk, Hq * D:], "dk, dv")


def test_bad_descriptors_contribute_nothing():
    Hq, Hkv, D, T = 4, 2, 64, 260
    good = [(0, 0, 100, 100, 50), (100, 100, 60, 60, 60)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=13)
    s, out, lse = _forward(qkv, good, Hq, Hkv, D)
    want = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    for bad in ((-1, 0, 5, 5, 5), (0, -1, 5, 5, 5), (200, 200, 61, 61, 0), (200, 200, 5, 61, 0), (200, 200, -1, 5, 0),
                (200, 200, 5, 0, 0), (200, 200, 5, 4, 1), (200, 200, 5, 5, 6), (200, 200, 5, 5, -1),
                (2 ** 31 - 1, 0, 2 ** 31 - 1, 5, 0), (0, 2 ** 31 - 1, 1, 2 ** 31 - 1, 0)):
        for at in (0, 1, 2):
            seqs = torch.tensor(good[:at] + [bad] + good[at:], dtype=torch.int32, device=DEV)
            d = _backward(dout, qkv, out, lse, seqs, Hq, Hkv, D, flags=mot.DEV_BAD_SEQUENCE)
            assert_bitwise(d, want, str(bad))


def test_many_sequences():
    # more descriptors than a warp's lanes and than any table of fixed size, ragged
    Hq, Hkv, D = 2, 1, 64
    lens = [1 + (i * 7) % 13 for i in range(333)]
    seqs, at = [], 0
    for i, n in enumerate(lens):
        seqs.append((at, at, n, n, (i * 3) % (n + 1)))
        at += n
    qkv, dout = _inputs(at, Hq, Hkv, D, seed=14)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D)


def test_long_sequences_among_many():
    # a prompt with latents that see its keys and a sequence that sees some of them, alone and beside more sequences than a table in
    # shared memory holds: the lists of work are made in another way, the bits are the same
    Hq, Hkv, D, T = 7, 1, 128, 1600
    few = [(0, 0, 1100, 1100, 900), (1100, 0, 300, 1100, 0), (1400, 200, 50, 333, 20)]
    many = [(1450 + i, 1450 + i, 1, 1, i % 2) for i in range(100)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=19)
    s, out, lse = _forward(qkv, few, Hq, Hkv, D)
    want = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    _check(want, dout, qkv, out, lse, few, Hq, Hkv, D)
    for seqs in (few + many, many[:40] + few + many[40:], many + few):
        s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
        d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
        assert_bitwise(d[:1450], want[:1450], f"{len(seqs)} sequences")
        _check(d[1450:, :], dout[1450:], qkv[1450:], out[1450:], lse[:, 1450:], [(q - 1450, k - 1450, *x) for q, k, *x in many],
               Hq, Hkv, D)


@pytest.mark.parametrize("Hq,Hkv,D,n", [(6, 2, 64, 1400), (4, 1, 64, 1250), (2, 2, 128, 1100), (2, 1, 128, 1281),
                                         (8, 1, 128, 1500), (12, 1, 64, 1500), (16, 2, 64, 1100)])
def test_shares_of_long_sequences(Hq, Hkv, D, n):
    # tiles whose blocks are shared by one CTA to sixteen, of whole and of few rows
    seqs = [(7, 7, n, n, n - 300), (n + 7, 900, 60, 60, 0)]
    qkv, dout = _inputs(n + 80, Hq, Hkv, D, seed=n)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D)
    assert_bitwise(d, _backward(dout, qkv, out, lse, s, Hq, Hkv, D), "again")


def test_short_sequences_over_few_keys():
    # many sequences' queries in one tile of keys: its blocks are shared out over all of them
    Hq, Hkv, D, keys = 8, 1, 64, 9
    seqs, at = [(0, 0, keys, keys, keys)], keys
    for i in range(70):
        n = 1 + i * 37 % 150
        seqs.append((at, 0, n, keys, 0))
        at += n
    qkv, dout = _inputs(at, Hq, Hkv, D, seed=29)
    for some in (seqs, seqs[:50]):
        s, out, lse = _forward(qkv, some, Hq, Hkv, D)
        d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
        _check(d, dout, qkv, out, lse, some, Hq, Hkv, D)


def test_two_graphs_with_one_workspace():
    Hq, Hkv, D = 7, 1, 128
    ws, graphs = _ws(700, Hq, Hkv, D, 70), []
    for T, seqs in ((700, [(0, 0, 700, 700, 500)]), (210, [(3 * i, 3 * i, 3, 3, 1) for i in range(70)])):
        qkv, dout = _inputs(T, Hq, Hkv, D, seed=T)
        s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
        want, got, graph = _backward(dout, qkv, out, lse, s, Hq, Hkv, D), torch.full_like(qkv, 7.0), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mot.mot_joint_attention_backward(dout, qkv, out, lse, s, Hq, Hkv, D, ws, dqkv=got)
        graphs.append((graph, got, want, (dout, qkv, out, lse, s)))
    for i in (0, 1, 1, 0, 1):
        graph, got, want, _ = graphs[i]
        got.fill_(7.0)
        graph.replay()
        assert_bitwise(got, want, f"graph {i}")
    assert mot.mot_device_status(ws) == 0


@pytest.mark.parametrize("n", [63, 64, 65, 128])
def test_where_the_table_of_sequences_ends(n):
    Hq, Hkv, D = 4, 2, 64
    seqs = [(3 * i, 3 * i, 3, 3, i % 4) for i in range(n)] + [(3 * n, 0, 20, 3 * n, 0)]
    qkv, dout = _inputs(3 * n + 20, Hq, Hkv, D, seed=n)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    _check(d, dout, qkv, out, lse, seqs, Hq, Hkv, D)


def test_layer_sampled_rows():
    # a whole layer's pack: sampled rows against the golden of their own (heads of one group)
    Hq, Hkv, D, T = 28, 4, 128, 2500
    seqs = [(10, 10, 1500, 1500, 1000), (1510, 1510, 900, 900, 900)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=15)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    d = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    G = Hq // Hkv
    for g in (0, 3):  # one KV head at a time is a smaller problem of its own
        cols = list(range(g * G * D, (g + 1) * G * D)) + list(range((Hq + g) * D, (Hq + g + 1) * D)) + \
            list(range((Hq + Hkv + g) * D, (Hq + Hkv + g + 1) * D))
        _check(d[:, cols], dout[:, g * G * D:(g + 1) * G * D], qkv[:, cols], out[:, g * G * D:(g + 1) * G * D],
               lse[g * G:(g + 1) * G], seqs, G, 1, D)


def test_streams_and_graphs():
    Hq, Hkv, D, T = 4, 2, 64, 333
    seqs = [(0, 0, 200, 200, 120), (200, 200, 133, 133, 133)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=16)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    want = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    other, od = _inputs(T, Hq, Hkv, D, seed=17)
    _, oout, olse = _forward(other, seqs, Hq, Hkv, D)
    owant = _backward(od, other, oout, olse, s, Hq, Hkv, D)
    # two calls at once, on streams of their own and with workspaces of their own
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [_ws(T, Hq, Hkv, D, 2) for _ in streams]
    d = [torch.full_like(qkv, 7.0) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        mot.mot_joint_attention_backward(dout, qkv, out, lse, s, Hq, Hkv, D, ws[0], dqkv=d[0], stream=streams[0])
        mot.mot_joint_attention_backward(od, other, oout, olse, s, Hq, Hkv, D, ws[1], dqkv=d[1], stream=streams[1])
    torch.cuda.synchronize()
    assert_bitwise(d[0], want, "stream 0")
    assert_bitwise(d[1], owant, "stream 1")
    # captured forward and backward, replayed on new contents of the same tensors
    x, do, o, l, dd = qkv.clone(), dout.clone(), out.clone(), lse.clone(), torch.full_like(qkv, 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mot.mot_joint_attention_lse(x, s, Hq, Hkv, D, ws[0], out=o, lse=l)
        mot.mot_joint_attention_backward(do, x, o, l, s, Hq, Hkv, D, ws[0], dqkv=dd)
    x.copy_(other)
    do.copy_(od)
    graph.replay()
    assert_bitwise(dd, owant, "replayed")
    x.copy_(qkv)
    do.copy_(dout)
    graph.replay()
    assert_bitwise(dd, want, "replayed again")
    assert mot.mot_device_status(ws[0]) == 0


def test_default_buffers_and_refusals():
    Hq, Hkv, D, T = 4, 2, 64, 70
    seqs = [(0, 0, 60, 60, 30)]
    qkv, dout = _inputs(T, Hq, Hkv, D, seed=18)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    ws = _ws(T, Hq, Hkv, D, 1)
    d = mot.mot_joint_attention_backward(dout, qkv, out, lse, s, Hq, Hkv, D, ws)
    assert not d[60:].any() and d[:60].any()
    good = dict(dout=dout, qkv=qkv, out=out, lse=lse, seqs=s, ws=ws, dqkv=torch.empty_like(qkv))

    def call(**kw):
        a = {**good, **kw}
        return mot.mot_joint_attention_backward(a["dout"], a["qkv"], a["out"], a["lse"], a["seqs"], Hq, Hkv, D, a["ws"],
                                                dqkv=a["dqkv"])

    for name, t in good.items():
        for bad in (7, t.double(), t.cpu(), t.unsqueeze(0)):
            with pytest.raises((TypeError, ValueError), match=name):
                call(**{name: bad})
    for name in ("dout", "out", "lse", "dqkv"):
        with pytest.raises(ValueError):
            call(**{name: good[name][:, :-8].contiguous()})
    with pytest.raises(ValueError, match="contiguous"):
        call(dout=dout.t().contiguous().t())
    with pytest.raises(mot.MotError):
        call(ws=ws[:-16].contiguous())


def _room_for(gb):
    if torch.cuda.mem_get_info()[0] < gb * 2 ** 30:
        pytest.skip(f"needs {gb} GB of free memory")


def test_rows_past_32_bit_offsets():
    # the last rows of a pack of more than 2^31 values: the same bits as in a pack of their own
    Hq, Hkv, D, n = 28, 4, 128, 333
    _room_for(40)
    T = 2 ** 31 // ((Hq + 2 * Hkv) * D) + 2 * n
    seqs = [(0, 0, 200, 200, 150), (200, 0, 133, 200, 0)]
    qkv, dout = _inputs(n, Hq, Hkv, D, seed=23)
    s, out, lse = _forward(qkv, seqs, Hq, Hkv, D)
    want = _backward(dout, qkv, out, lse, s, Hq, Hkv, D)
    big, bd, bo = (torch.zeros((T, x.shape[1]), dtype=torch.bfloat16, device=DEV) for x in (qkv, dout, out))
    bl = torch.zeros((Hq, T), device=DEV)
    big[-n:], bd[-n:], bo[-n:], bl[:, -n:] = qkv, dout, out, lse
    at = T - n
    ws = _ws(T, Hq, Hkv, D, 2)
    moved = torch.tensor([(q + at, k + at, *x) for q, k, *x in seqs], dtype=torch.int32, device=DEV)
    d = mot.mot_joint_attention_backward(bd, big, bo, bl, moved, Hq, Hkv, D, ws, dqkv=torch.full_like(big, 7.0))
    assert mot.mot_device_status(ws) == 0
    assert_bitwise(d[-n:], want, "the last rows")
    assert bool((d[:1000] == 7.0).all()) and bool((d[-n - 1000:-n] == 7.0).all())
