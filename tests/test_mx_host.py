"""Host-side checks of the MXFP4 and dropout calls (no GPU): storage sizes,
and every refusal before a device is touched.  The pointers are fake and never
dereferenced; a launch with them would fault."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

P = ctypes.c_void_p
FAKE, ODD = P(0x10000), P(0x10008)
NULL, ALIGN, SHAPE, RANK, WORKSPACE, DTYPE, DROPOUT, MX_SHAPE = -1, -2, -3, -4, -5, -12, -13, -14
OVERLAP = -15


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_15_b200 as q
    from bit_nf4_quantized_15_b200 import build
    build.build()
    return q


def _t(q, rows, cols, codes=0x1000, scales=0x2000):
    return ctypes.byref(q.mx.qlora_mx_tensor(codes, scales, rows, cols))


def _d(q, p=0.1, offset_dev=None):
    return ctypes.byref(q.mx.qlora_dropout_config(p, 1, 2, offset_dev))


def test_storage_bytes(q):
    assert q.mx_storage_bytes(128, 128) == (8192, 512)
    assert q.mx_storage_bytes(129, 160) == (129 * 80, 2 * 2 * 512)
    assert q.mx_storage_bytes(1, 32) == (16, 512)
    for bad in ((0, 32), (1, 0), (1, 48), (1 << 25, 32), (1, 1 << 25)):
        with pytest.raises(q.QLoRAError):
            q.mx_storage_bytes(*bad)


def test_quantise_and_dequant_refusals(q):
    L = q.lib()
    t = _t(q, 4, 64)
    assert L.qlora_mx_quantize(None, 0, 4, 64, 0, t, None, None) == NULL
    assert L.qlora_mx_quantize(FAKE, 0, 4, 64, 0, None, None, None) == NULL
    assert L.qlora_mx_quantize(FAKE, 0, 4, 64, 0, _t(q, 4, 64, codes=None), None, None) == NULL
    assert L.qlora_mx_quantize(FAKE, 3, 4, 64, 0, t, None, None) == DTYPE
    assert L.qlora_mx_quantize(FAKE, 0, 4, 48, 0, t, None, None) == MX_SHAPE
    assert L.qlora_mx_quantize(FAKE, 0, 0, 64, 0, t, None, None) == MX_SHAPE
    assert L.qlora_mx_quantize(FAKE, 0, 48, 64, 1, t, None, None) == MX_SHAPE       # blocks along 48 rows
    assert L.qlora_mx_quantize(FAKE, 0, 64, 12, 1, t, None, None) == MX_SHAPE
    assert L.qlora_mx_quantize(ODD, 0, 4, 64, 0, t, None, None) == ALIGN
    assert L.qlora_mx_quantize(FAKE, 0, 4, 64, 0, _t(q, 4, 64, scales=0x2004), None, None) == ALIGN
    assert L.qlora_mx_dequant(t, None, 0, None) == NULL
    assert L.qlora_mx_dequant(t, FAKE, 1, None) == DTYPE
    assert L.qlora_mx_dequant(_t(q, 4, 40), FAKE, 0, None) == MX_SHAPE
    assert L.qlora_mx_dequant(t, ODD, 0, None) == ALIGN


def test_matmul_refusals(q):
    L = q.lib()
    a, b = _t(q, 4, 64), _t(q, 16, 64)
    assert L.qlora_mx_matmul(None, b, FAKE, 0, None, None) == NULL
    assert L.qlora_mx_matmul(a, b, None, 0, None, None) == NULL
    assert L.qlora_mx_matmul(a, b, FAKE, 1, None, None) == DTYPE
    assert L.qlora_mx_matmul(a, _t(q, 16, 96), FAKE, 0, None, None) == MX_SHAPE
    assert L.qlora_mx_matmul(a, _t(q, 12, 64), FAKE, 0, None, None) == MX_SHAPE
    assert L.qlora_mx_matmul(_t(q, 0, 64), b, FAKE, 0, None, None) == MX_SHAPE
    assert L.qlora_mx_matmul(a, b, ODD, 0, None, None) == ALIGN
    assert L.qlora_mx_matmul(a, _t(q, 16, 64, codes=0x1008), FAKE, 0, None, None) == ALIGN


def test_dropout_refusals(q):
    L = q.lib()
    assert L.qlora_dropout(None, 0, 8, _d(q), FAKE, None) == NULL
    assert L.qlora_dropout(FAKE, 0, 8, None, FAKE, None) == NULL
    assert L.qlora_dropout(FAKE, 7, 8, _d(q), FAKE, None) == DTYPE
    assert L.qlora_dropout(FAKE, 0, -1, _d(q), FAKE, None) == SHAPE
    for p in (-0.1, 1.0, 2.0, float("nan"), 1 - 2.0 ** -18):
        assert L.qlora_dropout(FAKE, 0, 8, _d(q, p), FAKE, None) == DROPOUT
    assert L.qlora_dropout(FAKE, 0, 8, _d(q, 0.1, 0x1004), FAKE, None) == ALIGN
    assert L.qlora_dropout(FAKE, 0, 8, _d(q), ODD, None) == ALIGN
    assert L.qlora_dropout(FAKE, 0, 0, _d(q), FAKE, None) == 0


def test_linear_refusals(q):
    L = q.lib()
    big = 1 << 40

    def fwd(X=FAKE, M=4, w=_t(q, 32, 64), L1=FAKE, L2=FAKE, r=16, drop=None, Y=FAKE, T=FAKE, ws=FAKE, n=big):
        return L.qlora_mx_linear_fwd(X, M, w, L1, L2, r, 1.0, drop, Y, T, ws, n, None, None)

    assert fwd(X=None) == NULL and fwd(w=None) == NULL and fwd(Y=None) == NULL and fwd(ws=None) == NULL
    assert fwd(L1=None) == NULL and fwd(L2=None) == NULL and fwd(T=None) == NULL
    assert fwd(r=12) == RANK and fwd(r=136) == RANK and fwd(r=-8) == RANK
    assert fwd(M=0) == MX_SHAPE and fwd(w=_t(q, 12, 64)) == MX_SHAPE and fwd(w=_t(q, 32, 72)) == MX_SHAPE
    assert fwd(X=ODD) == ALIGN and fwd(T=ODD) == ALIGN and fwd(drop=_d(q, 1.5)) == DROPOUT

    def bwd(dY=FAKE, X=FAKE, M=4, T=FAKE, wt=_t(q, 64, 32), N=32, K=64, L1=FAKE, L2=FAKE, r=16, drop=None, dX=FAKE,
            dL1=FAKE, dL2=FAKE, ws=FAKE, n=big):
        return L.qlora_mx_linear_bwd(dY, X, M, T, wt, N, K, L1, L2, r, 1.0, drop, dX, dL1, dL2, ws, n, None, None)

    assert bwd(dY=None) == NULL and bwd(ws=None) == NULL and bwd(wt=None) == NULL
    assert bwd(X=None) == NULL and bwd(T=None) == NULL and bwd(L1=None) == NULL
    assert bwd(r=0) == RANK                                   # adapter gradients without an adapter
    assert bwd(N=40, wt=_t(q, 64, 40)) == MX_SHAPE            # no backward form: N % 32
    assert bwd(wt=_t(q, 32, 64)) == MX_SHAPE                  # the forward's form in its place
    assert bwd(M=0) == MX_SHAPE
    assert bwd(dL1=ODD) == ALIGN and bwd(drop=_d(q, -1.0)) == DROPOUT


def test_workspace_bytes(q):
    n = q.mx_linear_workspace_bytes
    assert n(16, 4096, 4096) > 0 and n(16, 4096, 4096, 16) > n(16, 4096, 4096)
    for bad in ((0, 64, 64, 16), (4, 60, 64, 16), (4, 64, 80, 16), (4, 64, 64, 12)):
        with pytest.raises(q.QLoRAError):
            n(*bad)


def test_binding_refuses_what_is_not_a_cuda_tensor(q):
    X = torch.zeros((4, 64), dtype=torch.bfloat16)
    t = q.MXTensor(torch.zeros(128, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64)
    for call in (lambda: q.mx_quantize(X), lambda: q.dropout(X, 0.1, 1), lambda: q.mx_dequant(t),
                 lambda: q.mx_matmul(t, t), lambda: q.mx_linear_fwd(X, q.MXWeight(t)),
                 lambda: q.mx_linear_bwd(X, X, None, q.MXWeight(t))):
        with pytest.raises(q.QLoRAError):
            call()
    for p, seed, off in ((0.1, -1, 0), (0.1, 0, -1), (0.1, 1 << 64, 0)):
        with pytest.raises(q.QLoRAError):
            q.Dropout(p, seed, off).config(X.device)


def test_workspace_never_falls_with_the_tokens(q):
    """One buffer for the largest batch serves the smaller ones."""
    n = q.mx_linear_workspace_bytes
    for N, K, r in ((4096, 4096, 64), (1024, 1024, 128), (64, 22016, 8), (22016, 8192, 16), (96, 64, 128),
                    (4096, 64, 0)):
        sizes = [n(M, N, K, r) for M in [*range(1, 4097), *range(4097, 20000, 61)]]
        falls = [i + 1 for i in range(len(sizes) - 1) if sizes[i + 1] < sizes[i]]
        assert not falls, (N, K, r, falls[:5])


def test_units_runs_and_slots(tmp_path):
    """The kernels' shares of the work, replayed on the host."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "mx_plan_check")
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", os.path.join(root, "bit_nf4_quantized_15_b200", "csrc"),
                    os.path.join(root, "tests", "mx_plan_check.cpp"), "-o", exe], check=True, capture_output=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout
    assert int(out.stdout.split("plans=")[1].split()[0]) > 20000


def test_overlapping_outputs_are_refused(q):
    """dX over an operand that a later gradient reads; dropout over a part of
    its input."""
    L = q.lib()
    M, N, K = 4, 32, 64
    p = lambda at: P(0x100000 + at)  # noqa: E731

    def bwd(dX, dL1=p(0x5000), dL2=p(0x6000)):
        return L.qlora_mx_linear_bwd(p(0), p(0x1000), M, p(0x2000), _t(q, K, N), N, K, p(0x3000), p(0x4000), 16, 1.0,
                                     None, dX, dL1, dL2, p(0x8000), 1 << 40, None, None)

    for at in (0x1000, 0x1000 + 2 * M * K - 16, 0x1000 - 2 * M * K + 16):   # X: all of it, its end, its start
        assert bwd(p(at)) == bwd(p(at), dL2=None) == OVERLAP
    assert bwd(p(0)) == bwd(p(0), dL1=None) == bwd(p(2 * M * N - 16)) == OVERLAP    # dY
    for n, dtype, size in ((64, 0, 2), (64, 1, 2), (64, 2, 4)):
        for step in (16, size * n - 16):
            assert L.qlora_dropout(p(0x400), dtype, n, _d(q), p(0x400 + step), None) == OVERLAP
            assert L.qlora_dropout(p(0x400), dtype, n, _d(q), p(0x400 - step), None) == OVERLAP
    assert b"overlap" in L.qlora_status_string(OVERLAP)


def test_seeds_and_offsets_are_whole_numbers(q):
    """A fraction was cut to another seed's mask."""
    for seed, off in ((1.5, 0), (2.0, 0), (0, 0.5), ("1", 0), (None, 0)):
        with pytest.raises(q.QLoRAError):
            q.Dropout(0.1, seed, off).config(torch.device("cpu"))
    c = q.Dropout(0.1, torch.tensor(7).item(), (1 << 64) - 1).config(torch.device("cpu"))
    assert (c.seed, c.offset, c.offset_dev) == (7, (1 << 64) - 1, None)


def test_status_words_the_gpu_cannot_write_are_refused(q):
    """A kernel would store to a host address, or past a narrower word."""
    dev = torch.device("cuda", 0)
    for status in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32, device="meta"), 0x1000):
        with pytest.raises(q.QLoRAError):
            q.mx._status_ptr(status, dev)
    cpu = torch.device("cpu")
    for status in (torch.zeros(1, dtype=torch.uint8), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(q.QLoRAError):
            q.mx._status_ptr(status, cpu)
    word = torch.zeros(1, dtype=torch.int32)
    assert q.mx._status_ptr(word, cpu) == word.data_ptr()
