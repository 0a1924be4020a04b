"""GPU parity of the MXFP4 calls and of dropout against the fp64 oracle
(oracle/mx.py).

Codes, scales, values and masks are exact.  A product's element is allowed
  half a bf16 step of the result (2^-8 relative; 0 for an fp32 result), plus
  the fp32 accumulation, (steps + 8) 2^-22 of the sum of the terms' sizes: the
  tensor cores add each step's products and the accumulator with at most one
  unit (2^-23) lost to truncation a step on either side,
and the LoRA term's operand RNbf16(s T) 2^-8 of its terms' sizes.  In dL1 and
dL2 the adapter operands are unrounded: the fp32 accumulation alone, in pieces
of at most 512 terms.
"""

import numpy as np
import pytest
import torch

from gpu_util import from_bits, to_f64
from oracle import mx as O

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8
UNIT = 2.0 ** -22
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _acc(k, step):
    return (-(-k // step) + 8) * UNIT


def _rand(shape, std, seed, dtype=torch.bfloat16):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(std)).to(dtype).cuda()


def _check_mx(t, x64):
    codes, s = O.mx_quantize(x64)
    assert (t.rows, t.cols) == x64.shape
    assert np.array_equal(t.scales.cpu().numpy(), O.mx_tile_scales(s))
    got = t.codes.cpu().numpy().reshape(t.rows, -1)
    got = np.stack([got & 15, got >> 4], 2).reshape(codes.shape)
    ok = np.repeat(s != 255, 32, axis=1)
    assert np.array_equal(got[ok], codes[ok])
    return codes, s


def _within(got, ref, bound, what):
    got = to_f64(got)
    assert np.isfinite(got).all(), what
    d = np.abs(got - ref)
    worst = np.unravel_index(np.argmax(d - bound), d.shape)
    assert (d <= bound).all(), f"{what}: {d[worst]:.3e} > {bound[worst]:.3e} at {worst}"


# ---------------------------------------------------------------- quantise
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("R,C", [(1, 32), (3, 96), (128, 128), (129, 4128), (777, 160), (257, 1024)])
def test_quantise_exact(lib, R, C, dtype):
    X = _rand((R, C), 1.0, R + C, DT[dtype])
    X[0, :32] = 0
    t = lib.mx_quantize(X)
    codes, s = _check_mx(t, to_f64(X))
    ref = O.mx_values(codes, s)
    assert np.array_equal(to_f64(lib.mx_dequant(t)), ref)
    assert np.array_equal(to_f64(lib.mx_dequant(t, dtype=torch.float32)), ref)
    assert lib.read_status() == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("R,C", [(32, 8), (96, 24), (128, 128), (160, 4104), (1056, 200)])
def test_quantise_transposed_exact(lib, R, C, dtype):
    X = _rand((R, C), 0.02, R * 3 + C, DT[dtype])
    t = lib.mx_quantize(X, transpose=True)
    codes, s = _check_mx(t, to_f64(X).T)
    assert np.array_equal(to_f64(lib.mx_dequant(t)), O.mx_values(codes, s))


@pytest.mark.parametrize("transpose", [False, True])
def test_quantise_special_values(lib, transpose):
    """Every tie, saturation, subnormals and the ends of the exponent range;
    a block with an Inf or NaN turns NaN and is reported."""
    X = torch.zeros((32, 256), dtype=torch.float32)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.5, 7.9])
    for i in range(32):
        scale = 2.0 ** float([-149, -140, -127, -126, -125, -100, -1, 0, 1, 100, 124, 125][i % 12])
        row = torch.cat([mids, -mids, torch.nextafter(mids, torch.tensor(9.0)), torch.tensor([4.0])])
        X[i, :28] = row * scale
        X[i, 32] = 2.0 ** -149
        X[i, 64:96] = -row[:32].sum() * scale if i % 12 < 10 else 1.0
        X[i, 96] = 3.4e38
    X = X if not transpose else X.t().contiguous()
    X = X.cuda()
    t = lib.mx_quantize(X, transpose=transpose)
    x64 = to_f64(X).T if transpose else to_f64(X)
    codes, s = _check_mx(t, x64)
    assert np.array_equal(to_f64(lib.mx_dequant(t, dtype=torch.float32)), O.mx_values(codes, s))
    assert lib.read_status() == 0
    for bad in (float("inf"), float("-inf"), float("nan")):
        Y = X.clone()
        Y.view(-1)[7 if not transpose else 7 * X.shape[1]] = bad
        t = lib.mx_quantize(Y, transpose=transpose)
        v = to_f64(lib.mx_dequant(t))
        assert np.isnan(v[0, :32]).all() and np.isfinite(v[1:]).all() and np.isfinite(v[0, 32:]).all()
        assert lib.read_status() == -7


# ---------------------------------------------------------------- product
MATMULS = [(1, 8, 32), (1, 128, 64), (3, 136, 4096), (16, 64, 96), (17, 136, 160), (32, 1032, 2048), (33, 200, 256),
           (64, 1000, 288), (65, 8, 512), (128, 264, 1056), (129, 128, 2080), (256, 256, 256), (257, 520, 320),
           (300, 2056, 1568), (1000, 264, 4128), (513, 3000, 416),
           (2300, 2312, 416), (2433, 2184, 64), (4100, 1288, 2336), (2304, 4864, 32)]   # CTA pairs, ragged


@pytest.mark.parametrize("M,N,K", MATMULS)
def test_matmul(lib, M, N, K):
    A, B = _rand((M, K), 1.0, M + K), _rand((N, K), 0.02, N + K + 1)
    a, b = lib.mx_quantize(A), lib.mx_quantize(B)
    A64, B64 = O.mx_rounded(to_f64(A)), O.mx_rounded(to_f64(B))
    ref, size = A64 @ B64.T, np.abs(A64) @ np.abs(B64).T
    f32 = lib.mx_matmul(a, b, dtype=torch.float32)
    _within(f32, ref, _acc(K, 64) * size, "fp32")
    out = lib.mx_matmul(a, b)
    _within(out, ref, HALF_BF16 * np.abs(ref) + _acc(K, 64) * size, "bf16")
    assert torch.equal(out, f32.bfloat16())
    assert torch.equal(out, lib.mx_matmul(a, b))
    assert lib.read_status() == 0


def test_matmul_writes_its_output_alone(lib):
    """Rows and bytes around an output that ends inside a tile stay."""
    M, N, K = 37, 200, 96
    a, b = lib.mx_quantize(_rand((M, K), 1, 1)), lib.mx_quantize(_rand((N, K), 1, 2))
    buf = torch.full((M * N + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[2048:2048 + M * N].view(M, N)
    lib.mx_matmul(a, b, out=out)
    assert torch.equal(out, lib.mx_matmul(a, b))
    assert (buf[:2048] == 7).all() and (buf[2048 + M * N:] == 7).all()


def test_matmul_nan_and_zero_blocks(lib):
    A, B = _rand((40, 512), 1, 3), _rand((136, 512), 1, 4)
    A[5, 70] = float("nan")
    A[9] = 0
    out = lib.mx_matmul(lib.mx_quantize(A), lib.mx_quantize(B))
    assert lib.read_status() == -7
    assert torch.isnan(out[5]).all() and (out[9] == 0).all()
    keep = [i for i in range(40) if i != 5]
    assert torch.isfinite(out[keep]).all()


def test_matmul_extreme_scales(lib):
    """Blocks of very different size in one sum, down to scale byte 0."""
    A, B = torch.zeros((20, 256)), torch.zeros((72, 256))
    rng = np.random.default_rng(8)
    for t in (A, B):
        e = rng.integers(-120, 60, (t.shape[0], 8))
        t.copy_(torch.from_numpy((rng.standard_normal((t.shape[0], 8, 32)) * 2.0 ** e[:, :, None]).reshape(t.shape)))
    A, B = A.cuda(), B.cuda()
    A64, B64 = O.mx_rounded(to_f64(A)), O.mx_rounded(to_f64(B))
    got = lib.mx_matmul(lib.mx_quantize(A), lib.mx_quantize(B), dtype=torch.float32)
    size = np.abs(A64) @ np.abs(B64).T
    # below the smallest normal number the accumulator may flush: 256 terms of at most 2^-126
    _within(got, A64 @ B64.T, _acc(256, 64) * size + 256 * 2.0 ** -126, "extreme scales")


# ---------------------------------------------------------------- dropout
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,p,seed,offset", [(1, 0.5, 1, 0), (7, 0.25, 2, 1), (8, 0.0, 3, 0), (4099, 0.1, 1 << 40, 3),
                                             (65536, 0.9, (1 << 64) - 1, (1 << 64) - 1), (1 << 20, 0.05, 5, 1 << 33)])
def test_dropout_exact(lib, n, p, seed, offset, dtype):
    X = _rand((n,), 1.0, n, DT[dtype])
    out = lib.dropout(X, p, seed, offset)
    keep = O.dropout_keep(n, p, seed, offset)
    x = X.float() * torch.tensor(O.dropout_scale(p), dtype=torch.float32)
    ref = torch.where(torch.from_numpy(keep).cuda(), x, 0.0).to(X.dtype)
    assert torch.equal(out, ref)
    Y = X.clone()
    lib.dropout(Y, p, seed, offset, out=Y)
    assert torch.equal(Y, out)


def test_dropout_drops_non_finite_and_reads_its_offset_on_the_device(lib):
    X = torch.full((4096,), float("nan"), device="cuda")
    keep = torch.from_numpy(O.dropout_keep(4096, 0.5, 11, 40)).cuda()
    out = lib.dropout(X, 0.5, 11, 40)
    assert torch.equal(torch.isnan(out), keep) and (out[~keep] == 0).all()
    off = torch.tensor([38], dtype=torch.int64, device="cuda")
    X.fill_(1.0)
    g = torch.cuda.CUDAGraph()
    lib.dropout(X, 0.5, 11, off)
    with torch.cuda.graph(g):
        out = lib.dropout(X, 0.5, 11, off)
    for o in (38, 40, 41):
        off.fill_(o)
        g.replay()
        assert torch.equal(out != 0, torch.from_numpy(O.dropout_keep(4096, 0.5, 11, o)).cuda())


# ----------------------------------------------------------------- linear
def _problem(lib, M, N, K, r, seed):
    X, W = _rand((M, K), 1.0, seed), _rand((N, K), 0.02, seed + 1)
    L1 = _rand((K, r), K ** -0.5, seed + 2) if r else None
    L2 = _rand((r, N), 0.05, seed + 3) if r else None
    return X, lib.mx_weight(W, backward=N % 32 == 0), L1, L2, _rand((M, N), 0.01, seed + 4), to_f64(W)


LINEARS = [(1, 64, 64, 8, 0.0), (5, 160, 288, 16, 0.5), (16, 1056, 512, 64, 0.1), (33, 96, 4128, 24, 0.0),
           (64, 320, 96, 128, 0.25), (129, 544, 1056, 72, 0.1), (300, 128, 2080, 64, 0.05), (777, 288, 320, 128, 0.1),
           (520, 2080, 1056, 16, 0.0), (1100, 96, 64, 8, 0.5), (70, 64, 96, 0, 0.0),
           (2100, 2336, 2400, 64, 0.1), (2400, 2080, 2528, 128, 0.0), (2049, 2304, 2304, 8, 0.25)]   # CTA pairs


@pytest.mark.parametrize("M,N,K,r,p", LINEARS)
def test_linear(lib, M, N, K, r, p):
    X, w, L1, L2, dY, W64 = _problem(lib, M, N, K, r, seed=M + N + K)
    s = 16.0 / max(r, 1)
    drop = lib.Dropout(p, 77 + M, 5) if p else None
    mask = O.dropout_keep(M * K, p, 77 + M, 5).reshape(M, K) * O.dropout_scale(p) if p else np.ones((M, K))
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, s, dropout=drop)
    X64, What = to_f64(X), O.mx_rounded(W64)
    if not r:
        assert T is None
        assert torch.equal(Y, lib.mx_matmul(lib.mx_quantize(X), w.fwd))
        dX, dL1, dL2 = lib.mx_linear_bwd(dY, None, None, w)
        assert dL1 is None and dL2 is None
        assert torch.equal(dX, lib.mx_matmul(lib.mx_quantize(dY), w.bwd))
        return
    A, B = to_f64(L1), to_f64(L2)
    Yr, Tr = O.mx_linear_fwd(X64, What, A, B, s, mask)
    t_err = _acc(min(K, 512), 16) * 2 * (np.abs(X64 * mask) @ np.abs(A)) + 2.0 ** -24 * 8 * np.abs(Tr)
    _within(T, Tr, t_err, "T")
    size = np.abs(O.mx_rounded(X64)) @ np.abs(What).T + s * np.abs(Tr) @ np.abs(B)
    y_err = HALF_BF16 * (np.abs(Yr) + s * np.abs(Tr) @ np.abs(B)) + (_acc(K, 64) + _acc(r, 16)) * size \
        + s * t_err @ np.abs(B) * 1.01
    _within(Y, Yr, y_err * 1.01, "Y")
    if w.bwd is None:
        return
    dX, dL1, dL2 = lib.mx_linear_bwd(dY, X, T, w, L1, L2, s, dropout=drop)
    dY64, T64, Wt = to_f64(dY), to_f64(T), O.mx_rounded(W64.T)
    dXr, dL1r, dL2r = O.mx_linear_bwd(dY64, X64, T64, Wt, A, B, s, mask)
    dTr = s * dY64 @ B.T
    dt_err = s * _acc(min(N, 512), 16) * 2 * (np.abs(dY64) @ np.abs(B).T) + 2.0 ** -24 * 8 * np.abs(dTr)
    lora = np.abs(dTr) @ np.abs(A).T * mask
    size = np.abs(O.mx_rounded(dY64)) @ np.abs(Wt).T + lora
    _within(dX, dXr, 1.01 * (HALF_BF16 * (np.abs(dXr) + lora) + (_acc(N, 64) + _acc(r, 16)) * size
                             + (dt_err @ np.abs(A).T) * mask), "dX")
    two = 3 * _acc(min(M, 512), 16) + 2.0 ** -22 * (M // 512)
    _within(dL1, dL1r, two * (np.abs(X64 * mask).T @ np.abs(dTr)) + np.abs(X64 * mask).T @ dt_err, "dL1")
    _within(dL2, dL2r, two * s * (np.abs(T64).T @ np.abs(dY64)), "dL2")
    assert lib.read_status() == 0


@pytest.mark.parametrize("M", [129, 250, 256])
def test_dL1_alike_with_the_mask_of_dX_and_without_dX(lib, M):
    """dL1 takes the mask's bits from the product of dX where that is wide
    enough to leave them, and evaluates them without it: bit for bit the same
    (one piece of the tokens either way).  The last columns end inside a tile."""
    N, K, r = 64, 9760, 32
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=31 + M)
    T = _rand((M, r), 1.0, 32).float()
    drop = lib.Dropout(0.4, 8, 9)
    dX, with_dX, _ = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop)
    none, alone, _ = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop, need_dX=False)
    assert dX is not None and none is None and torch.equal(with_dX, alone)
    assert lib.read_status() == 0


def test_linear_dropped_elements_get_the_base_gradient_alone(lib):
    """Where the mask drops an element of X, dX is the product's alone, bit
    for bit; elsewhere the adapter's term is there."""
    M, N, K, r = 200, 256, 512, 32
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=2)
    drop = lib.Dropout(0.3, 5, 6)
    full, _, _ = lib.mx_linear_bwd(dY, X, torch.zeros((M, r), device="cuda"), w, L1, L2 * 8, 2.0, dropout=drop)
    base = lib.mx_matmul(lib.mx_quantize(dY), w.bwd)
    keep = torch.from_numpy(O.dropout_keep(M * K, 0.3, 5, 6).reshape(M, K)).cuda()
    assert torch.equal(full[~keep], base[~keep])
    assert (full[keep] != base[keep]).float().mean() > 0.9


def test_linear_optional_outputs_and_workspace(lib):
    M, N, K, r = 100, 96, 160, 16
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=4)
    drop = lib.Dropout(0.1, 1, 2)
    ws = torch.full((lib.mx_linear_workspace_bytes(M, N, K, r),), 255, dtype=torch.uint8, device="cuda")
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, 0.5, dropout=drop)
    Y2, T2 = lib.mx_linear_fwd(X, w, L1, L2, 0.5, dropout=drop, ws=ws)
    assert torch.equal(Y, Y2) and torch.equal(T, T2)
    full = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop)
    ws.fill_(255)
    for i in range(3):
        flags = dict(need_dX=i == 0, need_dL1=i == 1, need_dL2=i == 2)
        part = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop, ws=ws, **flags)
        assert [p is not None for p in part] == [i == 0, i == 1, i == 2]
        assert torch.equal(part[i], full[i])


def test_linear_without_tokens(lib):
    X, w, L1, L2, dY, _ = _problem(lib, 2, 64, 96, 8, seed=1)
    Y, T = lib.mx_linear_fwd(X[:0], w, L1, L2, 0.5)
    assert Y.shape == (0, 64) and T.shape == (0, 8)
    dX, dL1, dL2 = lib.mx_linear_bwd(dY[:0], X[:0], T, w, L1, L2, 0.5)
    assert dX.shape == (0, 96) and not dL1.any() and not dL2.any()


def test_training_step_on_a_side_stream_and_in_a_graph(lib):
    """Forward and backward with dropout on another stream and from a captured
    graph give the bits of plain calls; new inputs in place give new results."""
    M, N, K, r = 260, 160, 320, 16
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=9)
    drop = lib.Dropout(0.1, 3, 4)

    def step():
        Y, T = lib.mx_linear_fwd(X, w, L1, L2, 0.5, dropout=drop)
        return (Y, T) + lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop)

    ref = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (20, 21):
        X.copy_(_rand((M, K), 1.0, seed))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(step(), out))


def test_one_step_of_training_runs_together(lib):
    """quantise -> forward -> backward -> optimizer on the adapters, as they
    are used: the step changes both adapters and the output."""
    M, N, K, r = 64, 128, 256, 16
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=12)
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, 1.0, dropout=lib.Dropout(0.1, 1, 0))
    _, dL1, dL2 = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 1.0, dropout=lib.Dropout(0.1, 1, 0))
    for p16, g in ((L1, dL1), (L2, dL2)):
        p = p16.float()
        m, v = torch.zeros_like(p), torch.zeros_like(p)
        before = p16.clone()
        lib.adamw_step(p, g, m, v, step=1, lr=1e-2, p_bf16=p16)
        assert (p16 != before).any() and torch.isfinite(p).all()
    Y2, _ = lib.mx_linear_fwd(X, w, L1, L2, 1.0)
    assert not torch.equal(Y, Y2) and lib.read_status() == 0


def test_expired_wait_is_reported_and_the_next_call_is_right(lib):
    a, b = lib.mx_quantize(_rand((40, 512), 1, 1)), lib.mx_quantize(_rand((200, 512), 1, 2))
    ref = lib.mx_matmul(a, b)
    lib.debug_stall_next_gemm(5_000_000)
    lib.mx_matmul(a, b)
    assert lib.read_status() == -8
    assert torch.equal(lib.mx_matmul(a, b), ref) and lib.read_status() == 0


# ------------------------------------------------- calls that are easy to break
def test_offsets_past_32_bits(lib):
    """More than 2^32 elements: the last rows are those of a small call."""
    R, C, tail = 131077, 32800, 300
    X = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    X[-tail:] = _rand((tail, C), 1.0, 5)
    t = lib.mx_quantize(X)
    small = lib.mx_quantize(X[-tail:].contiguous())
    assert torch.equal(t.codes.view(R, -1)[-tail:], small.codes.view(tail, -1))
    values = lib.mx_dequant(t)
    assert torch.equal(values[-tail:], lib.mx_dequant(small)) and not values[:-tail].any()
    del values, t, small
    out = lib.dropout(X, 0.5, 3, 1)
    kept = out[-tail:] != 0
    assert not out[:-tail].any()
    assert abs(kept.float().mean().item() - 0.5) < 5 * 0.5 / (tail * C) ** 0.5 + 1e-3
    # element i of the tail is element i of the whole: counters of one call after another
    q = np.arange((R * C - 8000) // 8, R * C // 8, dtype=np.uint64)
    lo, one = np.uint64(0xFFFFFFFF), np.ones_like(q)
    w = O.philox4x32([q & lo, q >> np.uint64(32), one, 0 * one], (3, 0))
    keep = np.stack([h for x in w for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], 1).reshape(-1) >= 32768
    last = out.view(-1)[-len(keep):].cpu().float().numpy() != 0
    assert np.array_equal(last, keep & (X.view(-1)[-len(keep):].cpu().float().numpy() != 0))
    del out, X
    M, N, K = 70001, 65536, 32
    a, b = lib.mx_quantize(_rand((M, K), 1.0, 6)), lib.mx_quantize(_rand((N, K), 1.0, 7))
    big = lib.mx_matmul(a, b)
    head = lib.mx_quantize(lib.mx_dequant(a)[-tail:].contiguous())
    assert torch.equal(big[-tail:], lib.mx_matmul(head, b))


def test_dropped_nan_reaches_no_adapter_sum(lib):
    """A NaN that the mask drops leaves T and dL1 finite; its row of Y is NaN
    through the quantised product.  A kept one makes its row of T NaN."""
    M, N, K, r, p = 130, 64, 96, 16, 0.5
    X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=6)
    keep = O.dropout_keep(M * K, p, 9, 9).reshape(M, K)
    row = 77
    dropped, kept = int(np.flatnonzero(~keep[row])[0]), int(np.flatnonzero(keep[row])[0])
    X[row, dropped] = float("nan")
    drop = lib.Dropout(p, 9, 9)
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, 1.0, dropout=drop)
    assert torch.isfinite(T).all() and torch.isnan(Y[row]).all() and torch.isfinite(Y[:row]).all()
    _, dL1, dL2 = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 1.0, dropout=drop)
    assert torch.isfinite(dL1).all() and torch.isfinite(dL2).all()
    X[row, kept] = float("nan")
    _, T = lib.mx_linear_fwd(X, w, L1, L2, 1.0, dropout=drop)
    assert torch.isnan(T[row]).all() and torch.isfinite(T[row + 1:]).all()
    assert lib.read_status() == -7


@pytest.mark.parametrize("M", [3, 300, 2500])
def test_two_streams_and_two_graphs_at_once(lib, M):
    """Independent calls on two streams, and two captured graphs replayed in
    turn and together, give the bits of calls one after another."""
    N, K, r = 1056, 544, 40
    sets = [_problem(lib, M, N, K, r, seed=s) for s in (30, 40)]

    def step(i):
        X, w, L1, L2, dY, _ = sets[i]
        drop = lib.Dropout(0.2, 5, i)
        Y, T = lib.mx_linear_fwd(X, w, L1, L2, 0.5, dropout=drop)
        return (Y, T) + lib.mx_linear_bwd(dY, X, T, w, L1, L2, 0.5, dropout=drop)

    ref = [step(0), step(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = step(i)
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(ref[i], got[i]))
    graphs, outs = [], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(i))
        graphs.append(g)
    for _ in range(3):
        for i in (0, 1):
            streams[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(ref[i], outs[i]))


@pytest.mark.parametrize("r", range(8, 136, 8))
def test_every_rank(lib, r):
    """All ranks against the fp64 adapter sums (their operands are exact: the
    error is that of fp32 sums), with and without the pieces of 512 tokens."""
    for M, N, K in ((70, 96, 320), (1100, 64, 128)):
        X, w, L1, L2, dY, _ = _problem(lib, M, N, K, r, seed=r)
        Y, T = lib.mx_linear_fwd(X, w, L1, L2, 1.0)
        Tr = to_f64(X) @ to_f64(L1)
        assert np.linalg.norm(to_f64(T) - Tr) <= 2e-6 * np.linalg.norm(Tr)
        _, dL1, dL2 = lib.mx_linear_bwd(dY, X, T, w, L1, L2, 1.0)
        g1 = to_f64(X).T @ (to_f64(dY) @ to_f64(L2).T)
        g2 = to_f64(T).T @ to_f64(dY)
        assert np.linalg.norm(to_f64(dL1) - g1) <= 2e-6 * np.linalg.norm(g1)
        assert np.linalg.norm(to_f64(dL2) - g2) <= 2e-6 * np.linalg.norm(g2)


def test_binding_refusals(lib):
    """Shapes, types, layouts and devices that a call does not take."""
    X, w, L1, L2, dY, _ = _problem(lib, 8, 64, 96, 16, seed=3)
    Y, T = lib.mx_linear_fwd(X, w, L1, L2, 1.0)
    E = lib.QLoRAError
    bad = [lambda: lib.mx_quantize(X[:, :48].contiguous()), lambda: lib.mx_quantize(X.t()),
           lambda: lib.mx_quantize(X.double()), lambda: lib.mx_quantize(X, transpose=True),
           lambda: lib.mx_quantize(X, out=lib.MXTensor.empty(9, 96)),
           lambda: lib.mx_dequant(w.fwd, dtype=torch.float16),
           lambda: lib.mx_matmul(lib.mx_quantize(X), w.bwd), lambda: lib.mx_matmul(w.fwd, lib.mx_quantize(X[:7])),
           lambda: lib.mx_linear_fwd(X.half(), w, L1, L2, 1.0), lambda: lib.mx_linear_fwd(X, w, L1, None, 1.0),
           lambda: lib.mx_linear_fwd(X, w, L1.t().contiguous(), L2, 1.0),
           lambda: lib.mx_linear_fwd(X, w, L1[:, :12].contiguous(), L2[:12].contiguous(), 1.0),
           lambda: lib.mx_linear_fwd(X, w, L1, L2, 1.0, dropout=lib.Dropout(1.0, 1)),
           lambda: lib.mx_linear_fwd(X, w, L1, L2, 1.0, ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: lib.mx_linear_fwd(X, w, L1, L2, 1.0, Y=Y.float()),
           lambda: lib.mx_linear_bwd(dY, X, T, lib.MXWeight(w.fwd), L1, L2, 1.0),
           lambda: lib.mx_linear_bwd(dY, X[:4], T, w, L1, L2, 1.0),
           lambda: lib.mx_linear_bwd(dY, X, T.bfloat16(), w, L1, L2, 1.0),
           lambda: lib.dropout(X.view(-1)[1:], 0.1, 1), lambda: lib.dropout(X, -0.1, 1),
           lambda: lib.dropout(X, 0.1, 1, torch.zeros(2, dtype=torch.int64, device="cuda")),
           lambda: lib.MXTensor(w.fwd.codes[:-1], w.fwd.scales, 64, 96).descriptor()]
    for i, call in enumerate(bad):
        with pytest.raises(E):
            call()
            pytest.fail(f"call {i} was not refused")
    assert lib.read_status() == 0
