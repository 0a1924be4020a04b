"""The MXFP4 linear layer, its products and dropout where they can go wrong:
small reductions that leave the LoRA term to carry the result, infinities, the
paths that long reductions take, buffers that the caller gives.

Bounds as in test_gpu_mx.py: half a bf16 step of a bf16 result, and one unit
lost to truncation a step of the tensor cores' fp32 sums."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from gpu_util import to_f64
from oracle import mx as O
from test_gpu_mx import HALF_BF16, _acc, _problem, _within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- the LoRA term's bits
@pytest.mark.parametrize("M,N,K,r,p", [(40, 352, 64, 8, 0.0), (1088, 256, 64, 16, 0.05), (257, 64, 96, 128, 0.0),
                                       (2304, 2304, 64, 8, 0.25), (2100, 2400, 32, 72, 0.1)])
def test_lora_term_keeps_sixteen_bits(lib, M, N, K, r, p):
    """Where the LoRA term is as large as the base product, Y and dX are off
    by the rounding of the result and by 2^-16 of the LoRA term's sizes, not by
    the 2^-8 of an operand rounded to bf16."""
    X, w, L1, L2, dY, W64 = _problem(lib, M, N, K, r, seed=M + r)
    s = 16.0 / r
    drop = lib.Dropout(p, 5, M) if p else None
    mask = O.dropout_keep(M * K, p, 5, M).reshape(M, K) * O.dropout_scale(p) if p else np.ones((M, K))
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, s, dropout=drop)
    dX, _, _ = lib.mx_linear_bwd(dY, X, T, w, L1, L2, s, dropout=drop)
    X64, dY64, A, B = to_f64(X), to_f64(dY), to_f64(L1), to_f64(L2)
    What, Wt = O.mx_rounded(W64), O.mx_rounded(W64.T)
    Yr, Tr = O.mx_linear_fwd(X64, What, A, B, s, mask)
    dXr, _, _ = O.mx_linear_bwd(dY64, X64, Tr, Wt, A, B, s, mask)
    two = _acc(2 * max(r, 16), 16)  # steps of both terms
    # T: a sum of K < 512 products and one rounding each of it, of s and of their product
    t_err = _acc(K, 16) * (np.abs(X64 * mask) @ np.abs(A)) + 2.0 ** -22 * np.abs(Tr)
    lora = s * np.abs(Tr) @ np.abs(B)
    size = np.abs(O.mx_rounded(X64)) @ np.abs(What).T + lora
    _within(Y, Yr, 1.01 * (HALF_BF16 * np.abs(Yr) + 2.0 ** -16 * lora + (_acc(K, 64) + two) * size
                           + s * t_err @ np.abs(B)), "Y")
    dTr = s * dY64 @ B.T
    dt_err = (5 * _acc(min(N, 512), 16)) * s * (np.abs(dY64) @ np.abs(B).T) + 2.0 ** -22 * np.abs(dTr)
    lora = (np.abs(dTr) @ np.abs(A).T) * mask
    size = np.abs(O.mx_rounded(dY64)) @ np.abs(Wt).T + lora
    _within(dX, dXr, 1.01 * (HALF_BF16 * np.abs(dXr) + 2.0 ** -16 * lora + (_acc(N, 64) + two) * size
                             + (dt_err @ np.abs(A).T) * mask), "dX")
    assert lib.read_status() == 0


@pytest.mark.parametrize("M,N", [(40, 352), (300, 9792)])
def test_infinite_adapter_gives_infinities(lib, M, N):
    """An infinity in L2 makes its column of Y +-Inf by the sign of s T, also
    where s T has no bits for a second term; one in L1 its column of dX."""
    K, r = 64, 16
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=3)
    L1[:, 3], L1[5, 3] = 0, 1.0           # T[:, 3] = X[:, 5]: a bf16, one term
    L2[3, 7], L2[9, 11] = float("inf"), float("-inf")
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, 1.0)
    assert torch.equal(T[:, 3], X[:, 5].float())
    inf = torch.tensor(float("inf"), device="cuda")
    assert torch.equal(Y[:, 7].float(), torch.copysign(inf, T[:, 3]))
    assert torch.equal(Y[:, 11].float(), torch.copysign(inf, -T[:, 9]))
    rest = [c for c in range(N) if c not in (7, 11)]
    assert torch.isfinite(Y[:, rest]).all()
    L2[3, 7] = L2[9, 11] = 0
    L1[20, 4] = float("inf")
    dX, _, _ = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 1.0)
    dT = to_f64(dY) @ to_f64(L2).T
    assert np.array_equal(to_f64(dX[:, 20]), np.copysign(np.inf, dT[:, 4]))
    assert torch.isfinite(dX[:, :20]).all() and torch.isfinite(dX[:, 21:]).all()


# ------------------------------------------------ non-finite values, gradients
def _same_non_finite(got, ref, what):
    """NaN and infinities where the formula has them, finite elsewhere."""
    got = to_f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)]), what
    assert np.isfinite(got[np.isfinite(ref)]).all(), what


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("M", [40, 1100])
@pytest.mark.parametrize("where", ["X", "dY", "T", "dT"])
def test_infinities_in_the_adapter_gradients(lib, where, M, p):
    """dL1 and dL2 of an infinite X, dY, T or dT are the formula's, whether the
    other side has bits in all three terms or in the first alone, in one piece
    of the tokens and in several."""
    N, K, r, s = 96, 160, 16, 0.5
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=M)
    L2[:, 5], L2[3] = 0.0, 0.0
    L2[3, 9] = 1.0                       # dT[:, 3] = s dY[:, 9]: a bf16
    T = torch.randn((M, r), generator=torch.Generator("cuda").manual_seed(M), device="cuda")
    T[:, 4] = T[:, 4].bfloat16().float()
    drop = lib.Dropout(p, 3, 4) if p else None
    keep = O.dropout_keep(M * K, p, 3, 4).reshape(M, K)
    m = M - 7
    if where == "X":
        X[m, int(np.flatnonzero(keep[m])[2])] = float("inf")
        X[m - 3, int(np.flatnonzero(keep[m - 3])[4])] = float("-inf")
    elif where == "dY":
        dY[m, 5] = float("-inf")         # where L2 has no column: dT meets 0 Inf
    elif where == "T":
        T[m, 2], T[m - 1, 4] = float("inf"), float("-inf")
    else:
        s, dY[m, 9], L2[6, 9] = 1e3, 1e30, 1e7   # s dT[m, 6] is past the largest fp32
    dX, dL1, dL2 = lib.mx_linear_bwd(dY, X, T, w, L1, L2, s, dropout=drop, need_dX=False)
    with np.errstate(all="ignore"):
        dT = to_f64(dY) @ to_f64(L2).T
        dT = (s * dT).astype(np.float32).astype(np.float64)
        Xm = np.where(keep, to_f64(X), 0.0)
        ref1, ref2 = Xm.T @ dT, s * to_f64(T).T @ to_f64(dY)
    _same_non_finite(dL1, ref1, "dL1")
    _same_non_finite(dL2, ref2, "dL2")
    assert not np.isfinite(ref1).all() or not np.isfinite(ref2).all()
    assert dX is None
    lib.read_status()


@pytest.mark.parametrize("M", [33, 1100])
def test_non_finite_operands_of_single_gradients_are_reported(lib, M):
    """Also where the call does not quantise dY (dL2 alone), and for X and T."""
    N, K, r = 96, 160, 24
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=M)
    T = torch.ones((M, r), device="cuda")
    lib.read_status()

    def status(dY=dY, X=X, T=T, **need):
        lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, need_dX=False, **need)
        return lib.read_status()

    def broken(t, value):
        t = t.clone()
        t[M - 1, 9] = value
        return t

    only1, only2 = dict(need_dL2=False), dict(need_dL1=False)
    assert status() == status(**only1) == status(**only2) == 0
    for value in (float("nan"), float("inf")):
        assert status(dY=broken(dY, value), **only2) == -7
        assert status(dY=broken(dY, value), **only1) == -7
        assert status(T=broken(T, value), **only2) == -7
        assert status(X=broken(X, value), **only1) == -7
        assert status(T=broken(T, value), **only1) == status(X=broken(X, value), **only2) == 0


# ------------------------------------------------------------ callers' buffers
def test_one_workspace_for_the_largest_batch(lib):
    """A workspace sized for the largest batch serves every smaller one, and
    what the calls before have left in it changes nothing."""
    N, K, r = 576, 1056, 64
    most = 2432
    X, w, L1, L2, dY, _ = _problem(lib, most, N, K, r, seed=8)
    ws = torch.full((lib.mx_linear_workspace_bytes(most, N, K, r),), 255, dtype=torch.uint8, device="cuda")
    for M in (most, 2304, 1100, 300, 40, 1):
        drop = lib.Dropout(0.2, M)
        Y, T = lib.mx_linear_fwd(X[:M], w, L1, L2, 0.5, dropout=drop)
        ref = (Y, T) + lib.mx_linear_bwd(dY[:M], X[:M], T, w, L1, L2, 0.5, dropout=drop)
        Y, T = lib.mx_linear_fwd(X[:M], w, L1, L2, 0.5, dropout=drop, ws=ws)
        got = (Y, T) + lib.mx_linear_bwd(dY[:M], X[:M], T, w, L1, L2, 0.5, dropout=drop, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(ref, got)), M
    assert lib.read_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_dropout_in_place_over_many_turns(lib, dtype):
    """out = X where every thread takes several groups of eight, and a tail."""
    X = torch.randn((1 << 24) + 13, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(dtype)
    out = lib.dropout(X, 0.3, 7, 1)
    assert lib.dropout(X, 0.3, 7, 1, out=X) is X
    assert torch.equal(X, out)


# ---------------------------------------------------------------- repetitions
@pytest.mark.parametrize("M,N,K,r", [(1, 4096, 8192, 16), (300, 1024, 4128, 128), (1000, 2080, 4096, 64)])
def test_cluster_sums_repeat_bit_for_bit(lib, M, N, K, r):
    """Many calls back to back, whose clusters start as those before leave:
    every one gives the first one's bits."""
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=5)
    ref = lib.mx_linear_fwd(X, w, L1, L2, 1.0)
    ref += lib.mx_linear_bwd(dY, X, ref[1], w, L1, L2, 1.0)
    runs = []
    for _ in range(100):
        Y, T = lib.mx_linear_fwd(X, w, L1, L2, 1.0)
        runs.append((Y, T) + lib.mx_linear_bwd(dY, X, T, w, L1, L2, 1.0))
    assert all(torch.equal(a, b) for run in runs for a, b in zip(ref, run))
    assert lib.read_status() == 0


def test_stall_request_belongs_to_its_thread(lib):
    """A request armed on one host thread is not taken by another's product."""
    a, b = (lib.mx_quantize(torch.randn((n, 512), device="cuda")) for n in (40, 200))
    ref = lib.mx_matmul(a, b)
    torch.cuda.synchronize()
    other = []

    def elsewhere():
        out = lib.mx_matmul(a, b)
        torch.cuda.synchronize()
        other.append((lib.read_status(), torch.equal(out, ref)))

    lib.debug_stall_next_gemm(5_000_000)
    t = threading.Thread(target=elsewhere)
    t.start()
    t.join()
    assert other == [(0, True)]
    lib.mx_matmul(a, b)
    assert lib.read_status() == -8
    assert torch.equal(lib.mx_matmul(a, b), ref) and lib.read_status() == 0


def test_first_cuda_call_of_a_host_thread(lib):
    """A thread whose first CUDA work is one of the calls."""
    M, N, K, r = 40, 128, 256, 16
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=6)
    nf4 = lib.quantize(torch.randn((N, K), device="cuda").bfloat16())

    def step(i):
        if i == 0:
            Y, T = lib.mx_linear_fwd(X, w, L1, L2, 0.5)
            return (Y, T) + lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5)
        if i == 1:
            return (lib.mx_matmul(lib.mx_quantize(X, transpose=False), w.fwd),)
        if i == 2:
            return (lib.mx_quantize(L2.t().contiguous(), transpose=True).codes,)
        Y, T = lib.linear_fwd(X, nf4, L1, L2, 0.5)
        return (Y, T) + lib.linear_bwd(dY, X, T, nf4, L1, L2, 0.5)

    ref = [step(i) for i in range(4)]
    torch.cuda.synchronize()
    got = {}
    for i in range(4):
        t = threading.Thread(target=lambda: got.__setitem__(i, step(i)))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert sorted(got) == [0, 1, 2, 3]
    assert all(torch.equal(a, b) for i in range(4) for a, b in zip(ref[i], got[i]))


def test_outputs_over_inputs_that_are_no_longer_read(lib):
    """Y over X, dX over X without dL1 and over dY without dL2 give the bits of
    separate buffers; where the operand is still read the call is refused."""
    M, N, r = 300, 544, 32
    X, w, L1, L2, dY, _ = _problem(lib, M, N, N, r, seed=14)
    drop = lib.Dropout(0.1, 5)
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, 0.5, dropout=drop)
    dX, dL1, dL2 = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop)

    def bwd(over, **need):
        g, x = dY.clone(), X.clone()
        return lib.mx_linear_bwd(g, x, T, w, L1, L2, 0.5, dropout=drop, dX=x if over == "X" else g, **need)

    a, _, b = bwd("X", need_dL1=False)
    assert torch.equal(a, dX) and torch.equal(b, dL2)
    a, b, _ = bwd("dY", need_dL2=False)
    assert torch.equal(a, dX) and torch.equal(b, dL1)
    for over in ("X", "dY"):
        with pytest.raises(lib.QLoRAError):
            bwd(over)
    x = X.clone()
    assert torch.equal(lib.mx_linear_fwd(x, w, L1, L2, 0.5, dropout=drop, Y=x)[0], Y)
    assert torch.equal(x, Y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matrices_without_rows(lib, dtype):
    """No tokens, no features: empty results of the right shapes, as the
    linear layer gives them."""
    X = torch.randn((3, 96), device="cuda").to(dtype)
    none = lib.mx_quantize(X[:0])
    assert (none.rows, none.cols) == (0, 96)
    assert lib.mx_dequant(none, dtype=dtype).shape == (0, 96)
    turned = lib.mx_quantize(torch.empty((64, 0), dtype=dtype, device="cuda"), transpose=True)
    assert (turned.rows, turned.cols) == (0, 64) and lib.mx_dequant(turned).shape == (0, 64)
    w = lib.mx_quantize(torch.randn((16, 96), device="cuda"))
    assert lib.mx_matmul(none, w, dtype=dtype).shape == (0, 16)
    assert lib.mx_matmul(w, none, dtype=dtype).shape == (16, 0)
    assert lib.dropout(X[:0], 0.5, 1).shape == (0, 96)
    for bad in (lambda: lib.mx_quantize(X[:0, :40].contiguous()), lambda: lib.mx_matmul(none, turned),
                lambda: lib.MXTensor.empty(0, 40), lambda: lib.MXTensor.empty(-1, 32),
                lambda: lib.mx_matmul(none, lib.mx_quantize(torch.randn((12, 96), device="cuda")))):
        with pytest.raises(lib.QLoRAError):
            bad()
    assert lib.read_status() == 0


# ------------------------------------------------------ long adapter reductions
@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("M,N,K,r", [(1, 64, 22016, 16), (1, 22016, 64, 128), (70, 4128, 22016, 64),
                                     (70, 22016, 4128, 8), (600, 64, 8224, 128), (1100, 4128, 4128, 64), (4500, 128, 96, 16)])
def test_long_adapter_sums_are_those_of_fp32(lib, M, N, K, r, p):
    """T, dL1 and dL2 over long reductions, by the kernels that finish a tile in
    a cluster and by those that leave partial sums, with dropout and without.

    The operands are exact, so the error is that of the sums.  In a piece of 512
    terms (32 steps) a step loses at most a unit of the running sum to
    truncation, half of one of 2^-23 to 2^-24 on average: 0.36 2^-23 |S_i|, with
    |S_i| growing as the root of the step 0.36 (2/3) 32 2^-23 = 0.92e-6 of the
    piece, toward zero.  Pieces are added with rounding (2^-24 each time, up to 43
    of them, at random: 0.3e-6).  A sum of 4128 terms in one piece would lose
    seven times that.  dL1 has dT's error on top of its own."""
    g = torch.Generator("cuda").manual_seed(M + N + K)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    X, dY = rnd(M, K).bfloat16(), (rnd(M, N) * 0.01).bfloat16()
    L1, L2 = (rnd(K, r) * K ** -0.5).bfloat16(), (rnd(r, N) * 0.05).bfloat16()
    w = lib.mx_weight((rnd(N, K) * 0.02).bfloat16())
    drop = lib.Dropout(p, 9, M) if p else None
    m = 1.0
    if p:
        m = torch.from_numpy(O.dropout_keep(M * K, p, 9, M).reshape(M, K)).cuda().double() * O.dropout_scale(p)
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, 0.5, dropout=drop)
    dX, dL1, dL2 = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop)
    alone = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop, need_dX=False)
    Xm = X.double() * m
    refs = (Xm @ L1.double(), Xm.t() @ (0.5 * dY.double() @ L2.double().t()), 0.5 * T.double().t() @ dY.double())
    for got, ref, bound, what in ((T, refs[0], 1.25e-6, "T"),
                                  (dL1, refs[1], 2.5e-6, "dL1"), (dL2, refs[2], 1.25e-6, "dL2"),
                                  (alone[1], refs[1], 2.5e-6, "dL1 alone"), (alone[2], refs[2], 1.25e-6, "dL2 alone")):
        err = float((got.double() - ref).norm() / ref.norm())
        assert err <= bound, f"{what}: {err:.2e}"
    assert torch.isfinite(Y).all() and torch.isfinite(dX).all() and lib.read_status() == 0


# ------------------------------------------------------- offsets on the device
@pytest.mark.parametrize("M,N,K,r", [(1, 64, 96, 8), (40, 96, 160, 16), (300, 2080, 544, 128), (2100, 2336, 2400, 64)])
def test_linear_reads_its_offset_on_the_device(lib, M, N, K, r):
    """Dropout with its offset in a CUDA tensor: each kernel that evaluates the
    mask reads it when it runs, eagerly and from one captured graph."""
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=M)
    off = torch.tensor([3], dtype=torch.int64, device="cuda")

    def step(offset):
        drop = lib.Dropout(0.3, 11, offset)
        Y, T = lib.mx_linear_fwd(X, w, L1, L2, 0.5, dropout=drop)
        both = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop)
        return (Y, T) + both + lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop, need_dX=False)[1:]

    refs = {o: step(o) for o in (3, 4, (1 << 40) + 1)}
    assert not torch.equal(refs[3][0], refs[4][0])
    for o in refs:
        off.fill_(o)
        assert all(torch.equal(a, b) for a, b in zip(step(off), refs[o]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(off)
    for o in refs:
        off.fill_(o)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, refs[o])), o
    assert lib.read_status() == 0


# ------------------------------------------------------------- given outputs
@pytest.mark.parametrize("M", [5, 300, 1100])
def test_outputs_go_to_the_buffers_given(lib, M):
    """Y, T, dX, dL1 and dL2 in the caller's memory, all of it and nothing else."""
    N, K, r = 96, 160, 24
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=M + 1)
    drop = lib.Dropout(0.2, 2)

    def inside(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 128,), 3.0, dtype=dtype, device="cuda")
        bufs.append((buf, n))
        return buf[64:64 + n].view(shape)

    bufs = []
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, 0.5, dropout=drop)
    grads = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop)
    y, t = inside((M, N), torch.bfloat16), inside((M, r), torch.float32)
    got = lib.mx_linear_fwd(X, w, L1, L2, 0.5, dropout=drop, Y=y, T=t)
    assert got[0] is y and got[1] is t and torch.equal(y, Y) and torch.equal(t, T)
    outs = [inside((M, K), torch.bfloat16), inside((K, r), torch.float32), inside((r, N), torch.float32)]
    got = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop, dX=outs[0], dL1=outs[1], dL2=outs[2])
    assert all(a is b for a, b in zip(got, outs)) and all(torch.equal(a, b) for a, b in zip(got, grads))
    for buf, n in bufs:
        assert (buf[:64] == 3).all() and (buf[64 + n:] == 3).all()


def test_gradients_in_the_flat_buffer_of_data_parallelism(lib):
    """AdapterGrads' views as the gradients of two layers: each writes its own
    part of the flat buffer, which is what a collective then sums."""
    from bit_nf4_quantized_15_b200.data_parallel import AdapterGrads
    M, r, shapes = 520, 16, [(96, 160), (320, 64)]
    grads = AdapterGrads(shapes, r)
    parts = []
    for i, (N, K) in enumerate(shapes):
        X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=i)
        Y, T = lib.mx_linear_fwd(X, w, L1, L2, 0.5)
        _, a, b = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5)
        parts += [a.reshape(-1), b.reshape(-1)]
        lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dL1=grads.dL1[i], dL2=grads.dL2[i])
    assert torch.equal(grads.flat, torch.cat(parts))
    assert grads.all_reduce() is grads


# ---------------------------------------------------------------- fp32 products
@pytest.mark.parametrize("M,N,K", [(16, 1024, 22016), (40, 22016, 8192), (130, 9600, 4160), (512, 8192, 22016),
                                   (2304, 2312, 8224)])
def test_fp32_product_of_blocks_of_many_sizes(lib, M, N, K):
    """Blocks over 2^24 : 1 in size, where the order of the sum matters: the
    pieces of 2048 terms are 32 steps each, so the error is as in
    test_long_adapter_sums_are_those_of_fp32 (0.92e-6 and the rounding of at most
    11 additions)."""
    g = torch.Generator("cuda").manual_seed(K + M)

    def mixed(rows):
        x = torch.randn((rows, K // 32, 32), generator=g, device="cuda")
        e = torch.rand((rows, K // 32, 1), generator=g, device="cuda") * 24 - 12
        return lib.mx_quantize((x * torch.exp2(e)).reshape(rows, K))

    a, b = mixed(M), mixed(N)
    got = lib.mx_matmul(a, b, dtype=torch.float32)
    ref = lib.mx_dequant(a, torch.float32).double() @ lib.mx_dequant(b, torch.float32).double().t()
    err = float((got.double() - ref).norm() / ref.norm())
    assert err <= 1.25e-6, f"{err:.2e}"
    assert torch.equal(got, lib.mx_matmul(a, b, dtype=torch.float32))
    assert lib.read_status() == 0


# ------------------------------------------------------- scales from elsewhere
def test_every_scale_byte_with_every_code(lib):
    """Also bytes that the quantiser never writes: values past the range are
    infinities, 255 is NaN."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))                 # 32 a row
    s = np.arange(256, dtype=np.uint8)[:, None]
    t = lib.MXTensor(torch.from_numpy(O.mx_pack(codes)).cuda(), torch.from_numpy(O.mx_tile_scales(s)).cuda(), 256, 32)
    with np.errstate(over="ignore"):
        ref = O.mx_values(codes, s).astype(np.float32)
    assert np.isinf(ref[253:255]).any() and not np.isinf(ref[:253]).any()
    for dtype in (torch.float32, torch.bfloat16):
        got = lib.mx_dequant(t, dtype=dtype).float().cpu().numpy()
        assert np.array_equal(got, ref, equal_nan=True), dtype


def test_product_of_large_scales_with_small_ones(lib):
    """Every pair of scale bytes whose product is a normal number."""
    rng = np.random.default_rng(4)
    s = np.arange(255, dtype=np.uint8)[:, None]
    a, b = (rng.integers(0, 16, (n, 32)).astype(np.uint8) for n in (255, 256))
    sb = np.minimum(np.arange(256), 254).astype(np.uint8)[:, None]
    A = lib.MXTensor(torch.from_numpy(O.mx_pack(a)).cuda(), torch.from_numpy(O.mx_tile_scales(s)).cuda(), 255, 32)
    B = lib.MXTensor(torch.from_numpy(O.mx_pack(b)).cuda(), torch.from_numpy(O.mx_tile_scales(sb)).cuda(), 256, 32)
    got = to_f64(lib.mx_matmul(A, B, dtype=torch.float32))
    A64, B64 = O.mx_values(a, s), O.mx_values(b, sb)
    ref, size = A64 @ B64.T, np.abs(A64) @ np.abs(B64).T
    e = s.astype(int) + sb.T.astype(int) - 254
    plain = (e >= -122) & (e <= 115)     # 32 products of at most 36 fit, and the least of 1/4 is normal
    assert np.array_equal(got[plain], ref[plain]) and plain.mean() > 0.6
    assert (size[plain] < 2.0 ** 127).all()


def test_asking_for_a_size_makes_no_context(lib):
    """A launcher may ask for workspace sizes before each rank picks its GPU."""
    code = ("import ctypes, bit_nf4_quantized_15_b200 as q\n"
            "assert q.mx_linear_workspace_bytes(16, 4096, 8192, 16) > 0\n"
            "assert q.mx_storage_bytes(128, 128) == (8192, 512)\n"
            "cu, flags, active = ctypes.CDLL('libcuda.so.1'), ctypes.c_uint(), ctypes.c_int(-1)\n"
            "assert cu.cuInit(0) == 0\n"
            "assert cu.cuDevicePrimaryCtxGetState(0, ctypes.byref(flags), ctypes.byref(active)) == 0\n"
            "print('active', active.value)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "active 0", out.stdout + out.stderr


def test_linear_past_32_bits_of_elements(lib):
    """More than 2^32 activations: the mask's counters, its bits, T, dX and the
    gradients of the last rows, the only ones that are not zero."""
    M, K, N, r, tail, s = 131077, 32800, 64, 8, 300, 0.5
    g = torch.Generator("cuda").manual_seed(2)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    X[-tail:] = rnd(tail, K).bfloat16()
    w = lib.mx_weight(rnd(N, K) * 0.02)
    L1, L2, dY = (rnd(K, r) * K ** -0.5).bfloat16(), (rnd(r, N) * 0.05).bfloat16(), rnd(M, N).bfloat16()
    drop = lib.Dropout(0.5, 3, 1)
    q = np.arange((M - tail) * K // 8, M * K // 8, dtype=np.uint64)
    lo, one = np.uint64(0xFFFFFFFF), np.ones_like(q)
    words = O.philox4x32([q & lo, q >> np.uint64(32), one, 0 * one], (3, 0))
    keep = np.stack([h for x in words for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], 1).reshape(-1) >= 32768
    keep = torch.from_numpy(keep.reshape(tail, K)).cuda()

    def near(got, ref, bound):
        err = float((got.double() - ref).norm() / ref.norm())
        assert err <= bound, f"{err:.2e}"

    Y, T = lib.mx_linear_fwd(X, w, L1, L2, s, dropout=drop)
    Xm, g64 = X[-tail:].double() * keep * 2, dY[-tail:].double()
    assert not T[:-tail].any() and not Y[:-tail].any()
    near(T[-tail:], Xm @ L1.double(), 1.5e-6)    # 0.92e-6, and 65 additions of pieces at random
    ref1, ref2 = Xm.t() @ (s * g64 @ L2.double().t()), s * T[-tail:].double().t() @ g64
    dX, dL1, dL2 = lib.mx_linear_bwd(dY, X, T, w, L1, L2, s, dropout=drop)
    near(dL1, ref1, 2.5e-6)
    near(dL2, ref2, 1.25e-6)
    base = lib.mx_matmul(lib.mx_quantize(dY[-tail:].contiguous()), w.bwd)
    assert torch.equal(dX[-tail:][~keep], base[~keep])
    assert (dX[-tail:][keep] != base[keep]).float().mean() > 0.9
    del dX, Y
    _, dL1, _ = lib.mx_linear_bwd(dY, X, T, w, L1, L2, s, dropout=drop, need_dX=False, need_dL2=False)
    near(dL1, ref1, 2.5e-6)
    assert lib.read_status() == 0
