"""The linear, grouped and SwiGLU operators where callers or values go astray:
offsets out of order, reports from several streams, the activations' far ends.
Tolerances as derived in test_gpu_linear.py."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import int4_quantized_expert_b200 as moe
from oracle import linear as ol
from tests.test_gpu_linear import check, f64, rnd, sum_tol

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# offsets out of order
# ---------------------------------------------------------------------------
def kept_ranges(off, n):
    """(begin, end) of each expert's rows; (0, 0) where the two offsets are no range of the rows, or
    one that overlaps an earlier range."""
    ranges = [(a, b) if 0 <= a <= b <= n else (0, 0) for a, b in zip(off, off[1:])]
    return [(a, b) if all(max(a, c) >= min(b, d) for c, d in ranges[:e]) else (0, 0) for e, (a, b) in enumerate(ranges)]


def overlapping_case(off, n, K, N):
    E, ranges = len(off) - 1, kept_ranges(off, n)
    x, w, dy = rnd(1, n, K), rnd(2, E, N, K, std=K ** -0.5), rnd(3, n, N)
    oc = torch.tensor(off, dtype=torch.int32, device="cuda")
    y = torch.full((n, N), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((n, K), 7.0, dtype=torch.bfloat16, device="cuda")
    assert moe.linear_device_status() == moe.Status.OK
    moe.grouped_linear(x.cuda(), w.cuda(), oc, out=y)
    assert moe.linear_device_status() == moe.Status.INVALID_ARG
    _, dw = moe.grouped_linear_backward(dy.cuda(), x.cuda(), w.cuda(), oc, dx=dx)
    assert moe.linear_device_status() == moe.Status.INVALID_ARG
    fx, fw, fdy = f64(x), f64(w), f64(dy)
    free = np.ones(n, bool)
    for e, (a, b) in enumerate(ranges):
        s = slice(a, b)
        free[s] = False
        check(y[s], fx[s] @ fw[e].T, sum_tol(K, np.abs(fx[s]) @ np.abs(fw[e]).T))
        check(dx[s], fdy[s] @ fw[e], sum_tol(N, np.abs(fdy[s]) @ np.abs(fw[e])))
        check(dw[e], fdy[s].T @ fx[s], sum_tol(b - a, np.abs(fdy[s]).T @ np.abs(fx[s])))
    free = torch.from_numpy(free).cuda()
    assert (y[free] == 7).all() and (dx[free] == 7).all()      # rows of no expert are left as they were


# Tiles whose contraction is split have a grid of as many as ranges that are apart
# can need: repeated ranges must not push the last expert's tiles out of it.
@pytest.mark.parametrize("off,n", [([0, 600, 0, 600, 640, 640], 640), ([0, 600, 0, 600, 0, 600, 640], 640),
                                   ([0, 48] * 8 + [48, 64], 64), ([0, 60] * 30 + [60, 64], 64),
                                   ([30, 64, 0, 30, 20, 64], 64), ([0, 128, 64, 192, 128, 256, 250, 300], 300),
                                   ([0, 9000, 0, 9000, 8000, 9001], 9001)])
@pytest.mark.parametrize("K,N", [(2056, 136), (136, 1032)])
def test_grouped_overlapping_ranges(off, n, K, N):
    if n > 1000:
        K, N = min(K, 264), min(N, 264)
    overlapping_case(off, n, K, N)


@pytest.mark.parametrize("off", [[0, 20, 10, 40, 64], [-5, 20, 20, 40, 64], [0, 20, 20, 40, 65], [64, 0, 64, 0, 64],
                                 [0, 20, 20, 40, 2 ** 31 - 1], [0, 20, 20, 40, -2 ** 31], [-2 ** 31, 2 ** 31 - 1, 0, 5, 64]])
def test_grouped_bad_offsets_row_by_row(off):
    overlapping_case(off, 64, 32, 48)


# ---------------------------------------------------------------------------
# the status word
# ---------------------------------------------------------------------------
def test_each_report_is_taken_once():
    """One thread makes a call that is reported, waits for it and queries; another queries all the
    while on its own stream.  Each report is returned to exactly one of them: none is lost between
    another query's reading and clearing, none is returned twice."""
    x, w = rnd(1, 64, 32).cuda(), rnd(2, 2, 48, 32).cuda()
    off = torch.tensor([0, 20, 65], dtype=torch.int32, device="cuda")     # one range past the rows: one report
    y = torch.empty(64, 48, dtype=torch.bfloat16, device="cuda")
    mine, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    assert moe.linear_device_status() == moe.Status.OK
    rounds, done, taken, wrong = 2000, threading.Event(), [0, 0], []

    def query(who, stream):
        s = moe.linear_device_status(stream)
        taken[who] += s == moe.Status.INVALID_ARG
        if s not in (moe.Status.OK, moe.Status.INVALID_ARG):
            wrong.append(s)

    def ask():
        while not done.is_set():
            query(1, other)

    t = threading.Thread(target=ask)
    t.start()
    try:
        for _ in range(rounds):
            moe.grouped_linear(x, w, off, out=y, stream=mine)
            mine.synchronize()
            query(0, mine)
    finally:
        done.set()
        t.join()
    assert not wrong and sum(taken) == rounds, (taken, wrong)
    assert moe.linear_device_status() == moe.Status.OK


# ---------------------------------------------------------------------------
# the activations' far ends
# ---------------------------------------------------------------------------
def every_bf16(lo, hi):
    """every bf16 value of magnitude lo .. hi, and its negative"""
    v = torch.arange(2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[(v.float() >= lo) & (v.float() <= hi)]
    return torch.cat([v, -v])


def through_slope(z, act):
    """act'(z): the bias gradient in fp32 of one row of ones"""
    n = -(-z.numel() // 8) * 8
    row = torch.zeros(1, n, dtype=torch.bfloat16)
    row[0, :z.numel()] = z
    row = row.cuda()
    _, _, db = moe.linear_backward(torch.ones_like(row), torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda"),
                                   torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda"), activation=act, preact=row,
                                   need_dx=False, need_dw=False, need_dbias=True, grad_dtype=torch.float32)
    return db[:z.numel()]


def test_gelu_slope_everywhere():
    """Within 3e-7, and in the negative tail within 3e-4 of itself (each from the fp32 evaluation of the
    formula; 2^-20 and 2^-11 leave the hardware's powers and reciprocals their part); values below 2^-122 may
    be flushed to 0 (a factor below 2^-126 is, times |z| < 16)."""
    z = every_bf16(2.0 ** -20, 100.0)
    got, want = f64(through_slope(z, moe.ACT_GELU)), ol.act_slope(f64(z), "gelu")
    assert (np.abs(got - want) <= 2.0 ** -20).all()
    tail = f64(z) < -1
    assert (np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -122)[tail].all()


def test_gelu_slope_of_infinite_values():
    inf, nan = float("inf"), float("nan")
    got = through_slope(torch.tensor([inf, -inf, 3e38, -3e38, nan, 0.0, -0.0, 33.0, -33.0]).bfloat16(), moe.ACT_GELU)
    assert got[[0, 2, 7]].eq(1).all() and got[[1, 3, 8]].eq(0).all() and got[4].isnan() and got[[5, 6]].eq(0.5).all()


def through_activation(z, act):
    """act(z) of bf16 values, by a product with the unit matrix (exact: one product with 1, the rest 0)"""
    x = torch.zeros(-(-z.numel() // 8), 8, dtype=torch.bfloat16)
    x.view(-1)[:z.numel()] = z
    return moe.linear(x.cuda(), torch.eye(8).bfloat16().cuda(), activation=act).view(-1)[:z.numel()]


def test_gelu_everywhere():
    """Within 2e-7 and 1.1e-3 of itself below -1 (the fit of Phi's logarithm in fp32; 2^-20 and 2^-9 leave the
    hardware's powers their part) before the one rounding to bf16; values below 2^-122 may be flushed to 0 (a
    factor below 2^-126 is, times |z| < 16)."""
    z = every_bf16(2.0 ** -20, 100.0)
    got, want = f64(through_activation(z, moe.ACT_GELU)), ol.act(f64(z), "gelu")
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20).all()
    tail = f64(z) < -1
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -9) * np.abs(want) + 2.0 ** -122)[tail].all()


def test_gelu_of_infinite_values():
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([inf, -inf, nan, 3e38, -3e38]).bfloat16()
    y = moe.linear(torch.ones(8, 8).bfloat16().cuda(), torch.zeros(8, 8).bfloat16().cuda(),
                   torch.cat([z, torch.zeros(3).bfloat16()]).cuda(), activation=moe.ACT_GELU)
    assert y[:, 0].eq(inf).all() and y[:, 1].eq(0).all() and y[:, 2].isnan().all()
    assert y[:, 3].eq(z[3].item()).all() and y[:, 4].eq(0).all()


def test_silu_everywhere():
    """The sigmoid is off by less than 2^-17 of itself (its exponent's rounding, 2^-18 at 88, the hardware's power
    and reciprocal); the slope s (1 + z (1 - s)) adds the roundings of a sum that is not below 1/2 for z < -2.
    Where the sigmoid is below 2^-126 it is 0."""
    z = every_bf16(2.0 ** -20, 100.0)
    fz = f64(z)
    got, want = f64(through_activation(z, moe.ACT_SILU)), ol.act(fz, "silu")
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(want) + 2.0 ** -119).all()
    got, want = f64(through_slope(z, moe.ACT_SILU)), ol.act_slope(fz, "silu")
    assert (np.abs(got - want) <= 2.0 ** -20 * (1 + np.abs(fz))).all()
    tail = fz < -2
    assert (np.abs(got - want) <= 2.0 ** -16 * np.abs(want) + 2.0 ** -119)[tail].all()


# ---------------------------------------------------------------------------
# the largest grouped calls
# ---------------------------------------------------------------------------
def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def test_grouped_weights_past_32_bits():
    """256 experts with 2^33 weights in all, the last experts' rows past 2^32 values."""
    E, K, N = 256, 4096, 8192
    counts = torch.zeros(E, dtype=torch.int64)
    counts[[0, 127, 128, 200, 255]] = torch.tensor([3, 70, 1, 300, 17])
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    n = int(off[-1])
    x, w, dy = normal(1, n, K), normal(2, E, N, K, std=K ** -0.5), normal(3, n, N)
    y = moe.grouped_linear(x, w, off.int().cuda())
    dx, dw = moe.grouped_linear_backward(dy, x, w, off.int().cuda())
    assert moe.linear_device_status() == moe.Status.OK
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        if s.start == s.stop:
            assert not dw[e].any()
            continue
        X, W, D = f64(x[s]), f64(w[e]), f64(dy[s])
        check(y[s], X @ W.T, sum_tol(K, np.abs(X) @ np.abs(W).T))
        check(dx[s], D @ W, sum_tol(N, np.abs(D) @ np.abs(W)))
        check(dw[e], D.T @ X, sum_tol(len(X), np.abs(D).T @ np.abs(X)))


@pytest.mark.parametrize("counts", [[1 << 20], [0, (1 << 20) - 7, 7, 0], [(1 << 20) // 256] * 256])
def test_grouped_most_rows(counts):
    n, E, K, N = sum(counts), len(counts), 24, 40
    off = np.concatenate([[0], np.cumsum(counts)])
    x, w, dy = normal(4, n, K), normal(5, E, N, K), normal(6, n, N)
    oc = torch.from_numpy(off).int().cuda()
    y = moe.grouped_linear(x, w, oc, out_dtype=torch.float32)
    dx, dw = moe.grouped_linear_backward(dy, x, w, oc, grad_dtype=torch.float32)
    assert moe.linear_device_status() == moe.Status.OK
    fx, fw, fdy = f64(x), f64(w), f64(dy)
    (rdx, rdw), (Sdx, Sdw) = ol.grouped_backward(fdy, fx, fw, off), ol.grouped_backward(abs(fdy), abs(fx), abs(fw), off)
    check(y, ol.grouped(fx, fw, off), sum_tol(K, ol.grouped(abs(fx), abs(fw), off)))
    check(dx, rdx, sum_tol(N, Sdx))
    check(dw, rdw, sum_tol(max(counts), Sdw))


# ---------------------------------------------------------------------------
# beside other work
# ---------------------------------------------------------------------------
def test_beside_products_on_another_stream():
    """Single tiles, pairs and split tiles on one stream, torch's products on another, at the same time: the same
    results as alone."""
    shapes = [(1, 4096, 4096), (40, 2048, 1024), (300, 1032, 2056), (3000, 520, 2056), (64, 256, 512)]
    args = [(normal(i, T, K), normal(i + 9, N, K, std=K ** -0.5)) for i, (T, K, N) in enumerate(shapes)]
    a, b = normal(30, 2048, 2048), normal(31, 2048, 2048)
    want, prod = [moe.linear(*v) for v in args], a @ b
    torch.cuda.synchronize()
    mine, other = torch.cuda.Stream(), torch.cuda.Stream()
    got, prods = [], []
    for _ in range(30):
        got.append([moe.linear(*v, stream=mine) for v in args])
        with torch.cuda.stream(other):
            prods.append(a @ b)
            prods.append(a[:64] @ b)
    torch.cuda.synchronize()
    assert moe.linear_device_status() == moe.Status.OK
    assert all(torch.equal(g, w) for row in got for g, w in zip(row, want))
    assert all(torch.equal(p, prod) for p in prods[::2])


def test_report_survives_an_error_of_another_call():
    """A query that fails because its stream is being captured leaves an error behind in this thread; the
    next query returns the report all the same."""
    code = """
import torch, int4_quantized_expert_b200 as moe
x, w = torch.zeros(64, 32).bfloat16().cuda(), torch.zeros(2, 48, 32).bfloat16().cuda()
bad = torch.tensor([0, 20, 65], dtype=torch.int32, device="cuda")
assert moe.linear_device_status() == moe.Status.OK
moe.grouped_linear(x, w, bad)
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.stream(s):
    g.capture_begin()
    assert moe.linear_device_status(s) == moe.Status.CUDA
    try:
        g.capture_end()
    except RuntimeError:
        pass
assert moe.linear_device_status() == moe.Status.INVALID_ARG
assert moe.linear_device_status() == moe.Status.OK
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300, cwd=os.path.dirname(os.path.dirname(__file__)))
