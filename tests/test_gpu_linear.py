"""linear, grouped_linear and swiglu with their gradients against the fp64 oracle.

Tolerances (derived, per element).  S is the sum of the products' magnitudes.
  sum   products of bf16 values are exact in fp32; each of C additions loses at
        most one fp32 step (2^-23) of a partial sum that is at most S, and a
        split contraction adds at most 8 partial sums: (C + 16) 2^-23 S
  act   |act'| <= 1.13 (GELU's largest slope, at sqrt 2) carries the sum's
        error; the activation itself is good to 2^-20 (1 + |z|)
  out   one rounding: 2^-8 (bf16) of the value, 2^-24 (fp32)
  dz    enters the products rounded to bf16; the reference rounds its fp64 dz.
        Where dz lies within its own error of a rounding border the other
        neighbour, one bf16 step away, is as right: that step's products are
        added to the bound.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import int4_quantized_expert_b200 as moe
from oracle import linear as ol
from oracle.ffn import bf16_round

pytestmark = pytest.mark.gpu

ACT = {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rnd(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.empty(*shape, dtype=torch.float32).normal_(0.0, std, generator=g).bfloat16()


def f64(t):
    return t.detach().cpu().double().numpy()


def sum_tol(C, S):
    return (C + 16) * 2.0 ** -23 * S


def check(got, ref, before):
    """got (a tensor) within its type's rounding of ref +- before"""
    u = U[got.dtype]
    got = f64(got)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= u * (np.abs(ref) + before) + before + 1e-37)
    assert not bad.any(), "%d of %d values off, first at %s: %r, reference %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], got[tuple(np.argwhere(bad)[0])], ref[tuple(np.argwhere(bad)[0])])


def forward_case(T, K, N, act, bias, residual, save, seed=0):
    x, w = rnd(seed, T, K), rnd(seed + 1, N, K, std=K ** -0.5)
    b = rnd(seed + 2, N) if bias else None
    r = rnd(seed + 3, T, N) if residual else None
    c = lambda t: None if t is None else t.cuda()
    got = moe.linear(c(x), c(w), c(b), activation=ACT[act], residual=c(r), save_preact=save)
    y, z = got if save else (got, None)
    assert moe.linear_device_status() == moe.Status.OK
    ry, rz = ol.linear(f64(x), f64(w), None if b is None else f64(b), act, None if r is None else f64(r))
    S = np.abs(f64(x)) @ np.abs(f64(w)).T + (0 if b is None else np.abs(f64(b)))
    tz = sum_tol(K, S)
    check(y, ry, 1.13 * tz + (0 if act in ("none", "relu") else 2.0 ** -20 * (1 + np.abs(rz))) + 2.0 ** -24 * np.abs(ry))
    if save:
        check(z, rz, tz)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 255, 257, 300, 513])
@pytest.mark.parametrize("K,N", [(8, 8), (72, 200), (520, 136)])
def test_linear_forward_sizes(T, K, N):
    forward_case(T, K, N, "silu", True, True, True, seed=T)


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("bias,residual,save", [(0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)])
def test_linear_forward_epilogues(act, bias, residual, save):
    forward_case(97, 136, 264, act, bias, residual, save, seed=7)
    forward_case(3, 2048, 264, act, bias, residual, save, seed=8)    # contraction split over a cluster


@pytest.mark.parametrize("T,K,N", [(1, 5120, 5120), (1, 16384, 256), (16, 5120, 1032), (64, 8192, 128), (200, 4096, 640),
                                   (1, 65536, 8), (2, 8, 65536), (5, 64, 19200)])
def test_linear_forward_few_rows_and_long_sums(T, K, N):
    forward_case(T, K, N, "none", True, True, False, seed=11)


# tiles of 16 to 192 rows whose contraction is split over up to 8 CTAs: rows
# around the tiles' ends, features around a block's, contractions that leave some
# CTAs a step more than others
@pytest.mark.parametrize("T", [1, 3, 4, 5, 17, 33, 47, 63, 79, 96, 111, 128, 130, 144, 159, 176, 191, 192, 193])
def test_linear_split_tiles(T):
    forward_case(T, 1096, 264, "gelu", True, True, True, seed=T)
    forward_case(T, 4104, 72, "none", False, True, False, seed=T + 1)


@pytest.mark.parametrize("T,K,N", [(100, 40, 3000), (192, 264, 1608), (3, 136, 5128), (1100, 72, 200), (2000, 8, 8)])
def test_linear_backward_split_tiles(T, K, N):
    backward_case(T, K, N, "silu", torch.bfloat16, seed=17)
    backward_case(T, N, K, "gelu", torch.float32, seed=18)


# tiles of 256 features shared by two CTAs: rows around their chunks' ends (32,
# 192, 256 and 320 rows, two accumulators from 257 on), features around 256,
# contractions around 16 and 64
@pytest.mark.parametrize("T", [225, 256, 257, 288, 289, 300, 320, 321, 500, 515, 640, 1000])
def test_linear_forward_pairs(T):
    forward_case(T, 72, 5128, "gelu", True, True, True, seed=T)


@pytest.mark.parametrize("T,K,N", [(129, 8, 9480), (700, 1032, 4104), (2100, 136, 1288), (4099, 200, 520), (1217, 328, 2824)])
def test_linear_pairs_sizes(T, K, N):
    forward_case(T, K, N, "none", False, True, False, seed=13)
    backward_case(T, N, K, "silu", torch.bfloat16, seed=14)
    backward_case(T, K, N, "relu", torch.float32, seed=15)


# tiles of 256 features whose contraction is split over two to four pairs of CTAs
@pytest.mark.parametrize("T,K,N", [(224, 4104, 3592), (256, 5120, 5120), (480, 5128, 2056), (700, 4104, 1544), (511, 1544, 264)])
def test_linear_forward_split_pairs(T, K, N):
    forward_case(T, K, N, "gelu", True, True, True, seed=19)


@pytest.mark.parametrize("T,K,N,act", [(250, 3080, 4104, "silu"), (8187, 1024, 1000, "relu"), (300, 520, 4104, "none")])
def test_linear_backward_split_pairs(T, K, N, act):
    backward_case(T, K, N, act, torch.bfloat16 if T < 400 else torch.float32, seed=20)


def test_linear_residual_in_place_and_repeat_calls():
    for T, K, N in ((5, 1024, 512), (700, 256, 520)):
        x, w, r = rnd(1, T, K).cuda(), rnd(2, N, K, std=K ** -0.5).cuda(), rnd(3, T, N).cuda()
        want = moe.linear(x, w, residual=r)
        assert torch.equal(want, moe.linear(x, w, residual=r))
        got = r.clone()
        assert moe.linear(x, w, residual=got, out=got) is got
        assert torch.equal(got, want)


def test_linear_extreme_values():
    """Infinite and NaN inputs stay in their own row and column; large and tiny
    pre-activations reach the activations' tails."""
    x, w = torch.zeros(70, 64).bfloat16(), torch.zeros(136, 64).bfloat16()
    x[:, 0] = torch.linspace(-30, 30, 70).bfloat16()
    w[:, 0] = 1
    x[7, 1] = float("inf")
    w[9, 2] = float("nan")
    for act in ACT:
        y = moe.linear(x.cuda(), w.cuda(), activation=ACT[act]).cpu().float()
        ok = torch.ones(70, 136, dtype=torch.bool)
        ok[7], ok[:, 9] = False, False
        assert y[:, 9].isnan().all()
        assert y[7].isnan().all()     # inf * 0 in every sum of the row
        ref = ol.act(f64(x[:, :1]), act).repeat(136, 1)
        got = y.double().numpy()
        m = ok.numpy()
        # absolute error 2^-20 (1 + |z|) as above; one bf16 rounding
        assert (np.abs(got - ref)[m] <= (2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * 31)[m]).all()


def backward_case(T, K, N, act, dtype, seed=0, need=(True, True, True)):
    x, w, dy, z = rnd(seed, T, K), rnd(seed + 1, N, K, std=N ** -0.5), rnd(seed + 2, T, N), rnd(seed + 3, T, N, std=1.5)
    got = moe.linear_backward(dy.cuda(), x.cuda(), w.cuda(), activation=ACT[act], preact=z.cuda() if act != "none" else None,
                              need_dx=need[0], need_dw=need[1], need_dbias=need[2], grad_dtype=dtype)
    assert moe.linear_device_status() == moe.Status.OK
    assert [g is not None for g in got] == list(need)
    dz = ol.linear_dz(f64(dy), f64(z), act)
    dzr = bf16_round(dz)
    # the slope's absolute error, as for the activation
    small = 2.0 ** -20 * (0 if act in ("none", "relu") else 1) * np.abs(f64(dy)) * (1 + np.abs(f64(z)))
    m, e = np.frexp(np.abs(dz) * 256)            # m in [1/2, 1): a bf16 step of dz is ulp = 2^(e - 16)
    ulp = np.ldexp(1.0, e - 16)
    off_border = np.abs(np.abs(dz) / ulp - np.floor(np.abs(dz) / ulp) - 0.5) * ulp
    flip = np.where(off_border <= small + 2.0 ** -18 * np.abs(dz), ulp, 0.0)
    dx, dw, db = ol.linear_backward(dzr, f64(x), f64(w))
    A, W, X = np.abs(dzr), np.abs(f64(w)), np.abs(f64(x))
    if need[0]:
        check(got[0], dx, sum_tol(N, A @ W) + flip @ W + small @ W)
    if need[1]:
        check(got[1], dw, sum_tol(T, A.T @ X) + flip.T @ X + small.T @ X)
    if need[2]:
        check(got[2], dz.sum(0), sum_tol(T, np.abs(dz).sum(0)) + small.sum(0))


@pytest.mark.parametrize("T", [1, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 129, 257, 530])
@pytest.mark.parametrize("K,N", [(8, 8), (200, 72), (136, 520)])
def test_linear_backward_sizes(T, K, N):
    backward_case(T, K, N, "gelu", torch.bfloat16, seed=T)


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("need", [(1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)])
def test_linear_backward_forms(act, dtype, need):
    backward_case(77, 264, 136, act, dtype, seed=5, need=tuple(map(bool, need)))


@pytest.mark.parametrize("T,K,N", [(1000, 128, 128), (4099, 64, 72), (3, 1024, 4096), (300, 2056, 1032)])
def test_linear_backward_splits_and_large(T, K, N):
    backward_case(T, K, N, "silu", torch.float32, seed=9)


def test_linear_gradient_against_differences():
    """The loss <y, dy> along a random direction of x, w and b, in the kernels
    themselves: both sides in bf16 outputs, so within the roundings of the sums
    over all outputs (2^-8 of their magnitudes, as random signs: 6 sigma)."""
    T, K, N, act = 64, 96, 80, "gelu"
    x, w, b, dy = rnd(1, T, K).cuda(), rnd(2, N, K, std=K ** -0.5).cuda(), rnd(3, N).cuda(), rnd(4, T, N).cuda()
    y, z = moe.linear(x, w, b, activation=ACT[act], save_preact=True)
    dx, dw, db = moe.linear_backward(dy, x, w, activation=ACT[act], preact=z, need_dbias=True, grad_dtype=torch.float32)
    ux, uw, ub = rnd(5, T, K).cuda().double(), rnd(6, N, K).cuda().double(), rnd(7, N).cuda().double()
    h = 1e-4

    def loss(s):   # the forward function in fp64 at the displaced point
        zz = (x.double() + s * ux) @ (w.double() + s * uw).T + (b.double() + s * ub)
        return (zz * torch.special.ndtr(zz) * dy.double()).sum().item()

    want = (loss(h) - loss(-h)) / (2 * h)
    terms = [(dx.double(), ux), (dw.double(), uw), (db.double(), ub)]
    got = sum((g * u).sum().item() for g, u in terms)
    # dz (a bf16 rounding, and z a bf16 rounding whose effect on the slope is at most 2^-8 |z| |act''| <= 2^-8 |z|)
    # carries up to 2 roundings into each term, dx one more
    dz = ol.linear_dz(f64(dy), f64(z), act)
    noise = 2.0 ** -8 * np.sqrt(sum(((np.abs(dz) * (np.abs(a)) ) ** 2).sum() for a in
                                    (f64(ux) @ f64(w).T, f64(x) @ f64(uw).T, f64(ub)[None] + 0 * dz)))
    noise_z = 2.0 ** -8 * np.sqrt(((np.abs(f64(dy) * f64(z)) * np.abs(f64(ux) @ f64(w).T + f64(x) @ f64(uw).T + f64(ub))) ** 2).sum())
    noise_dx = 2.0 ** -8 * np.sqrt(((f64(dx) * f64(ux)) ** 2).sum())
    assert abs(got - want) <= 6 * (noise + noise_z + noise_dx)


def test_linear_no_rows():
    w = rnd(1, 24, 16).cuda()
    x, dy = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    assert moe.linear(x, w).shape == (0, 24)
    dx, dw, db = moe.linear_backward(dy, x, w, need_dbias=True)
    assert dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    we = rnd(1, 3, 24, 16).cuda()
    assert moe.grouped_linear(x, we, off).shape == (0, 24)
    dx, dw = moe.grouped_linear_backward(dy, x, we, off)
    assert dx.shape == (0, 16) and (dw == 0).all()
    assert moe.swiglu(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")).shape == (0, 16)


# ---------------------------------------------------------------------------
COUNTS = {
    "one_row": [0, 1, 0, 0],
    "single": [300],
    "empty_ends": [0, 0, 5, 64, 0, 65, 130, 0],
    "odd": [1, 2, 3, 15, 16, 17, 31, 33, 47, 63, 64, 65],
    "long": [257, 513, 1, 0, 700],
    "many": [(7 * i * i) % 11 for i in range(256)],
}


def ragged(counts, before=0, after=0):
    off = np.concatenate([[0], np.cumsum(counts)]) + before
    return off.astype(np.int64), int(off[-1]) + after


def grouped_case(counts, K, N, y_dtype=torch.bfloat16, g_dtype=torch.bfloat16, before=0, after=0, seed=0):
    off, n = ragged(counts, before, after)
    E = len(counts)
    x, w, dy = rnd(seed, n, K), rnd(seed + 1, E, N, K, std=K ** -0.5), rnd(seed + 2, n, N)
    outside = np.ones(n, bool)
    outside[off[0]:off[-1]] = False
    x[outside] = float("nan")     # rows of no expert are not read
    dy[outside] = float("nan")
    xc, wc, dyc, oc = x.cuda(), w.cuda(), dy.cuda(), torch.from_numpy(off).int().cuda()
    y = torch.full((n, N), 7.0, dtype=y_dtype, device="cuda")
    assert moe.grouped_linear(xc, wc, oc, out_dtype=y_dtype, out=y) is y
    dx = torch.full((n, K), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dw = moe.grouped_linear_backward(dyc, xc, wc, oc, dx=dx, grad_dtype=g_dtype)
    assert moe.linear_device_status() == moe.Status.OK
    assert (y[torch.from_numpy(outside).cuda()] == 7).all() and (dx[torch.from_numpy(outside).cuda()] == 7).all()
    fx, fw, fdy, ins = f64(x), f64(w), f64(dy), torch.from_numpy(~outside).cuda()
    ry, (rdx, rdw) = ol.grouped(fx, fw, off), ol.grouped_backward(fdy, fx, fw, off)
    S, (Sdx, Sdw) = ol.grouped(abs(fx), abs(fw), off), ol.grouped_backward(abs(fdy), abs(fx), abs(fw), off)
    check(y[ins], ry[~outside], sum_tol(K, S[~outside]))
    check(dx[ins], rdx[~outside], sum_tol(N, Sdx[~outside]))
    check(dw, rdw, sum_tol(max(counts), Sdw))
    again = moe.grouped_linear_backward(dyc, xc, wc, oc, need_dx=False, grad_dtype=g_dtype)
    assert again[0] is None and torch.equal(again[1], dw)


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("K,N", [(8, 8), (136, 72), (264, 136)])
def test_grouped_sizes(name, K, N):
    grouped_case(COUNTS[name], K, N, seed=len(name))


@pytest.mark.parametrize("y_dtype,g_dtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
def test_grouped_types_and_rows_of_no_expert(y_dtype, g_dtype):
    grouped_case([40, 0, 130, 7], 136, 200, y_dtype, g_dtype, before=5, after=77, seed=3)
    grouped_case([2, 0, 0, 1], 1024, 264, y_dtype, g_dtype, before=1, after=3, seed=4)   # split contraction


def test_grouped_wide():
    grouped_case([3, 0, 70, 1, 0, 0, 9, 300], 2056, 1544, seed=6)


@pytest.mark.parametrize("counts", [[300, 257, 320, 321, 0, 640, 641, 1000, 31], [960, 961, 1, 0, 512, 288, 289, 1281],
                                    [256, 0, 255, 225, 224, 193, 192, 161, 700]])
@pytest.mark.parametrize("K,N", [(72, 2056), (1544, 264)])
def test_grouped_pairs(counts, K, N):
    grouped_case(counts, K, N, before=3, after=9, seed=len(counts))
    grouped_case(counts, K, N, torch.float32, torch.float32, seed=len(counts))


def test_grouped_neighbours_do_not_leak():
    """NaN in one expert's rows or weights stays in that expert's results."""
    counts, K, N = [37, 50, 29], 72, 136
    off, n = ragged(counts)
    x, w, dy = rnd(1, n, K), rnd(2, 3, N, K), rnd(3, n, N)
    oc = torch.from_numpy(off).int().cuda()
    want_y = moe.grouped_linear(x.cuda(), w.cuda(), oc)
    want_dx, want_dw = moe.grouped_linear_backward(dy.cuda(), x.cuda(), w.cuda(), oc)
    x[37:87], w[1], dy[37:87] = float("nan"), float("nan"), float("inf")
    y = moe.grouped_linear(x.cuda(), w.cuda(), oc)
    dx, dw = moe.grouped_linear_backward(dy.cuda(), x.cuda(), w.cuda(), oc)
    for got, want in ((y, want_y), (dx, want_dx)):
        assert torch.equal(got[:37], want[:37]) and torch.equal(got[87:], want[87:]) and not got[37:87].isfinite().any()
    assert torch.equal(dw[0], want_dw[0]) and torch.equal(dw[2], want_dw[2]) and not dw[1].isfinite().any()


def test_grouped_bad_offsets_are_reported():
    """An expert with offsets out of order or range counts as empty; the others' results are right."""
    x, w, dy = rnd(1, 64, 32).cuda(), rnd(2, 4, 48, 32).cuda(), rnd(3, 64, 48).cuda()
    good = torch.tensor([0, 20, 20, 40, 64], dtype=torch.int32, device="cuda")
    want, (wdx, wdw) = moe.grouped_linear(x, w, good), moe.grouped_linear_backward(dy, x, w, good)
    for bad, keep in (([0, 20, 10, 40, 64], (0, 3)), ([-5, 20, 20, 40, 64], (2, 3)), ([0, 20, 20, 40, 65], (0, 2)),
                      ([0, 20, 20, 40, 2 ** 31 - 1], (0, 2)), ([0, 20, 20, 40, -2 ** 31], (0, 2))):
        assert moe.linear_device_status() == moe.Status.OK
        oc = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y = moe.grouped_linear(x, w, oc)
        assert moe.linear_device_status() == moe.Status.INVALID_ARG
        dx, dw = moe.grouped_linear_backward(dy, x, w, oc)
        assert moe.linear_device_status() == moe.Status.INVALID_ARG
        for e in keep:
            s = slice(int(good[e]), int(good[e + 1]))
            if bad[1:3] == [20, 10] and e == 3:
                assert torch.equal(y[s], want[s])
            assert torch.equal(y[s], want[s]) or bad[2] == 10
            assert torch.equal(dw[e], wdw[e])


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,F", [(1, 8), (3, 72), (16, 8192), (333, 1032)])
def test_swiglu(n, F):
    gu, dh = rnd(1, n, 2 * F, std=2.0), rnd(2, n, F)
    if F > 8:
        gu[0, :4] = torch.tensor([100.0, -100.0, 30.0, -30.0]).bfloat16()
    h, d = moe.swiglu(gu.cuda()), moe.swiglu_backward(dh.cuda(), gu.cuda())
    g, u = np.split(f64(gu), 2, axis=1)
    # sigmoid, product: a few fp32 roundings of each factor; the slope's 1 + g (1 - s) to 2^-20 (1 + |g|)
    check(h, ol.swiglu(f64(gu)), 2.0 ** -20 * np.abs(g * u))
    small = 2.0 ** -20 * np.concatenate([np.abs(f64(dh) * u) * (1 + np.abs(g)), np.abs(f64(dh) * g)], axis=1)
    check(d, ol.swiglu_backward(f64(dh), f64(gu)), small)


# ---------------------------------------------------------------------------
def test_experts_forward_and_backward_together():
    """bf16 experts as they are run and trained: route, gather, the two grouped
    products with SwiGLU between them, the gate-weighted sum, and back."""
    T, D, F, E, k = 96, 256, 384, 8, 2
    x, wr = rnd(1, T, D).cuda(), rnd(2, E, D, std=0.05).cuda()
    w13, w2 = rnd(3, E, 2 * F, D, std=D ** -0.5).cuda(), rnd(4, E, D, F, std=F ** -0.5).cuda()
    dout = rnd(5, T, D).cuda()
    r = moe.route(x, wr, None, k)
    slots = r["perm"].long()
    xs, gates = x[slots // k].contiguous(), r["gates"].reshape(-1)[slots]
    gu = moe.grouped_linear(xs, w13, r["offsets"])
    h = moe.swiglu(gu)
    y = moe.grouped_linear(h, w2, r["offsets"], out_dtype=torch.float32)
    out = torch.zeros(T, D, device="cuda").index_add_(0, slots // k, y * gates[:, None])
    dy = (dout[slots // k].float() * gates[:, None]).bfloat16()
    dh, dw2 = moe.grouped_linear_backward(dy, h, w2, r["offsets"])
    dgu = moe.swiglu_backward(dh, gu)
    dxs, dw13 = moe.grouped_linear_backward(dgu, xs, w13, r["offsets"])
    dx = torch.zeros(T, D, device="cuda").index_add_(0, slots // k, dxs.float())
    assert moe.linear_device_status() == moe.Status.OK
    # the same layer in fp64 with autograd, every expert on its rows
    lx, l13, l2 = (t.double().requires_grad_() for t in (x, w13, w2))
    ref = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    ids = r["ids"].reshape(-1)
    g64 = r["gates"].reshape(-1).double()
    for e in range(E):
        s = (ids == e).nonzero()[:, 0]
        a, b = (lx[s // k] @ l13[e].T).chunk(2, dim=1)
        ref = ref.index_add(0, s // k, (torch.nn.functional.silu(a) * b) @ l2[e].T * g64[s, None])
    ref.backward(dout.double())
    # bf16 roundings on the way: gu, h | dy, dh, dgu: at most five of 2^-8 each, as 2-norms
    for got, want in ((out, ref.detach()), (dx, lx.grad), (dw13, l13.grad), (dw2, l2.grad)):
        assert (got.double() - want).norm() <= 5 * 2.0 ** -8 * want.norm()


def test_captured_and_replayed():
    """The whole chain in a CUDA graph: replays read the inputs' new contents."""
    E, K, N = 4, 264, 136
    x, w, dy = rnd(1, 90, K).cuda(), rnd(2, E, N, K).cuda(), rnd(3, 90, N).cuda()
    off = torch.tensor([0, 30, 30, 61, 90], dtype=torch.int32, device="cuda")
    w1, b1 = rnd(4, 64, N).cuda(), rnd(5, 64).cuda()

    def chain():
        y = moe.grouped_linear(x, w, off)
        o, z = moe.linear(y, w1, b1, activation=moe.ACT_GELU, save_preact=True)
        g = moe.linear_backward(o, y, w1, activation=moe.ACT_GELU, preact=z, need_dbias=True)
        return (y, o, z, *g, *moe.grouped_linear_backward(g[0], x, w, off), moe.swiglu(o))

    chain()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = chain()
    for seed, bounds in ((11, [0, 30, 30, 61, 90]), (12, [0, 1, 80, 80, 88])):
        x.copy_(rnd(seed, 90, K))
        off.copy_(torch.tensor(bounds, dtype=torch.int32))
        for t in outs:
            t.zero_()
        g.replay()
        want = chain()
        torch.cuda.synchronize()
        rows = bounds[-1]
        for got, ref in zip(outs[:3], want[:3]):
            assert torch.equal(got[:rows], ref[:rows])
        if rows == 90:
            for got, ref in zip(outs, want):
                assert torch.equal(got, ref)
    assert moe.linear_device_status() == moe.Status.OK


def test_two_streams_at_once():
    shapes = [(5, 2048, 512), (700, 264, 520)]
    args = [(rnd(i, T, K).cuda(), rnd(i + 5, N, K).cuda()) for i, (T, K, N) in enumerate(shapes)]
    want = [moe.linear(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(moe.linear(*args[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_waits_time_out_then_the_next_call_recovers():
    x, w = rnd(1, 300, 520).cuda(), rnd(2, 264, 520).cuda()
    one, wide = rnd(3, 1, 4096).cuda(), rnd(4, 128, 4096).cuda()
    dy = rnd(5, 300, 264).cuda()
    few, square = rnd(6, 256, 4096).cuda(), rnd(7, 3840, 4096).cuda()
    calls = [lambda: [moe.linear(x, w)], lambda: [moe.linear(one, wide)], lambda: [moe.linear(few, square)],
             lambda: [t for t in moe.linear_backward(dy, x, w)[:2]]]
    for call in calls:
        want = call()
        assert moe.linear_device_status() == moe.Status.OK
        moe.set_wait_limit(1)
        try:
            call()
            assert moe.linear_device_status() == moe.Status.TIMEOUT
        finally:
            moe.set_wait_limit(0)
        got = call()
        assert moe.linear_device_status() == moe.Status.OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    """A weight of 2^32 values: rows far into w, dx's sums over them, and dw's far rows."""
    T, K, N = 24, 65536, 65536
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, std=1.0: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)
    x, w, dy = r(T, K), r(N, K, std=K ** -0.5), r(T, N)
    rows = [0, 1, 32767, 32768, 40000, 65534, 65535]
    y = moe.linear(x, w)
    dx, dw, _ = moe.linear_backward(dy, x, w)
    assert moe.linear_device_status() == moe.Status.OK
    check(y[:, rows], f64(x) @ f64(w[rows]).T, sum_tol(K, np.abs(f64(x)) @ np.abs(f64(w[rows])).T))
    check(dw[rows], f64(dy[:, rows]).T @ f64(x), sum_tol(T, np.abs(f64(dy[:, rows])).T @ np.abs(f64(x))))
    cols = [0, 7, 32768, 65535]
    check(dx[:, cols], f64(dy) @ f64(w[:, cols]), sum_tol(N, np.abs(f64(dy)) @ np.abs(f64(w[:, cols]))))


@pytest.mark.parametrize("K,N", [(8, 16), (136, 8)])
def test_the_most_rows(K, N):
    T = 1 << 20
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s, std=1.0: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)
    x, w, dy = r(T, K), r(N, K), r(T, N)
    y = moe.linear(x, w)
    dx, dw, db = moe.linear_backward(dy, x, w, need_dbias=True, grad_dtype=torch.float32)
    assert moe.linear_device_status() == moe.Status.OK
    x, w, dy = (t.double() for t in (x, w, dy))
    for got, ref, S, C in ((y, x @ w.T, x.abs() @ w.abs().T, K), (dx, dy @ w, dy.abs() @ w.abs(), N),
                           (dw, dy.T @ x, dy.abs().T @ x.abs(), T), (db, dy.sum(0), dy.abs().sum(0), T)):
        u = U[got.dtype]
        tol = sum_tol(C, S)
        assert ((got.double() - ref).abs() <= u * (ref.abs() + tol) + tol).all()


def test_first_call_of_a_process_may_be_captured():
    code = """
import torch, int4_quantized_expert_b200 as moe
bf = dict(dtype=torch.bfloat16, device="cuda")
x, w, dy = torch.ones(300, 2048, **bf), torch.ones(3600, 2048, **bf), torch.ones(300, 3600, **bf)
one, off = torch.ones(1, 2048, **bf), torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y, t = moe.linear(x, w), moe.linear(one, w, activation=moe.ACT_RELU)
    dx, dw, db = moe.linear_backward(dy, x, w, activation=moe.ACT_GELU, preact=dy, need_dbias=True)
    z = moe.grouped_linear(x, w.view(2, 1800, 2048), off)
    h = moe.swiglu(y)
g.replay()
assert moe.linear_device_status() == 0
assert (y == 2048).all() and (t == 2048).all() and (z == 2048).all() and (h > 1e6).all() and dw.isfinite().all()
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300, cwd=os.path.dirname(os.path.dirname(__file__)))
