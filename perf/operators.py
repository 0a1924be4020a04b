"""Microscaled 4-bit operators and counter-based dropout: the cases they are measured on.

Four operators, next to the NF4 quantiser and the quantized linear layer of this package:

* ``quantize``: bf16, fp16 or fp32 to MXFP4 (E2M1 codes, one power-of-two scale for 32 elements) along the rows or,
  transposed, along the columns, and back to the values it stands for;
* ``matmul``: the product A.B^T of two MXFP4 tensors;
* ``linear_fwd`` / ``linear_bwd``: a LoRA linear layer whose frozen weight is MXFP4 and whose activations (forward) and
  upstream gradients (backward) are quantised on the way, with dropout on the adapter's input;
* ``dropout``: zeroes elements by a counter-based generator (Philox4x32-10), the mask never stored.

MXFP4 storage, which `prepare` makes and both sides read: codes uint8 [rows, cols / 2], element 2j in the low nibble; scales
uint8 E8M0 (2^(b - 127)) in tiles of 128 rows x 4 blocks, 512 bytes each, tiles of one row range consecutive; inside a
tile the scale of row i and block j is byte (i % 32) * 16 + (i // 32) * 4 + j.  Bytes outside the matrix are zero.
"""

import math

import torch

own = False

BLOCK = 32
BF16, F16, F32 = "bf16", "fp16", "fp32"
DTYPES = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
SIZES = {BF16: 2, F16: 2, F32: 4}
MAX_FLOPS = 2 * 8192 * 22016 * 8192


# ------------------------------------------------------------------- cases
def listed():
    return [
        # activations of a LLaMA-65B block, the operand of every product
        dict(name="quantize_8192x8192", op="quantize", rows=8192, cols=8192, dtype=BF16, transpose=False),
        # a LLaMA-7B gate weight in fp32, quantised along the output features for the backward product
        dict(name="quantize_t_11008x4096_f32", op="quantize", rows=11008, cols=4096, dtype=F32, transpose=True),
        # a LLaMA-65B attention projection on 8192 tokens, both sides in 4 bits
        dict(name="matmul_8192x8192x8192", op="matmul", M=8192, N=8192, K=8192),
        # sixteen decoded tokens through a LLaMA-65B up projection: the weight is read once
        dict(name="matmul_16x22016x8192", op="matmul", M=16, N=22016, K=8192),
        # ragged: rows that end inside a tile, columns that end inside a scale tile and inside a 64-wide step
        dict(name="matmul_1000x2056x1568", op="matmul", M=1000, N=2056, K=1568),
        # one decoded token through a 4096 x 4096 linear with a small adapter: latency
        dict(name="linear_fwd_1x4096x4096", op="linear_fwd", M=1, N=4096, K=4096, r=16, p=0.0),
        # a training forward of the LLaMA-7B gate with LoRA dropout
        dict(name="linear_fwd_4096x11008x4096_drop", op="linear_fwd", M=4096, N=11008, K=4096, r=64, p=0.1),
        # the largest forward: the LLaMA-65B gate on 8192 tokens
        dict(name="linear_fwd_8192x22016x8192", op="linear_fwd", M=8192, N=22016, K=8192, r=64, p=0.0),
        # the backward of the dropped LLaMA-7B gate
        dict(name="linear_bwd_4096x11008x4096_drop", op="linear_bwd", M=4096, N=11008, K=4096, r=64, p=0.1),
        # a ragged micro-batch in the backward, wide adapter
        dict(name="linear_bwd_777x2080x4128", op="linear_bwd", M=777, N=2080, K=4128, r=128, p=0.05),
        # dropout of the block's activations, as the adapter path of a linear layer sees it
        dict(name="dropout_8192x8192", op="dropout", n=8192 * 8192, dtype=BF16, p=0.1),
        # dropout of an odd fp32 vector
        dict(name="dropout_1048573_f32", op="dropout", n=1048573, dtype=F32, p=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["quantize", "matmul", "linear_fwd", "linear_bwd", "dropout"])
    if op == "quantize":
        t = rng.random() < 0.5
        while True:
            rows = _mult(rng, 32, 16384, 32) if t else _log(rng, 1, 16384)
            cols = _mult(rng, 8, 22016, 8) if t else _mult(rng, 32, 22016, 32)
            if rows * cols <= 1 << 27:
                return dict(op=op, rows=rows, cols=cols, dtype=rng.choice([BF16, BF16, F16, F32]), transpose=t)
    if op == "dropout":
        return dict(op=op, n=_log(rng, 1000, 1 << 27), dtype=rng.choice([BF16, BF16, F16, F32]),
                    p=rng.choice([0.05, 0.1, 0.25, 0.5]))
    while True:
        M = _log(rng, 1, 8192)
        N = _mult(rng, 64, 22016, 8 if op == "matmul" else 32)
        K = _mult(rng, 64, 22016, 32)
        if 2 * M * N * K <= MAX_FLOPS // 4 and N * K <= 8192 * 22016:
            break
    if op == "matmul":
        return dict(op=op, M=M, N=N, K=K)
    return dict(op=op, M=M, N=N, K=K, r=8 * _log(rng, 1, 16), p=rng.choice([0.0, 0.05, 0.1]))


# ------------------------------------------------- plain form: MXFP4 pieces
def _levels(device):
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=device)


def _quantize(x):
    """Codes (one a byte) [rows, cols] and E8M0 scale bytes [rows, cols / 32] of a matrix, blocks along its rows.

    The scale is 2^(floor(log2(max)) - 2) (not below 2^-127), an element the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6
    times the scale, ties to the even code, larger ones to 6."""
    x = x.float()
    b = x.reshape(x.shape[0], -1, BLOCK)
    expo = (b.abs().amax(2).contiguous().view(torch.int32) >> 23) & 255
    s = torch.where(expo == 255, expo, (expo - 2).clamp_min(0))
    v = torch.ldexp(b, (127 - s).unsqueeze(2))  # exact: a power of two
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    code = code + 8 * (v < 0).int()
    return code.reshape(x.shape).to(torch.uint8), s.to(torch.uint8)


def _pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def _tile_scales(s):
    """[rows, blocks] scale bytes to the tiled storage."""
    r, b = s.shape
    rt, bt = -(-r // 128), -(-b // 4)
    pad = s.new_zeros((rt * 128, bt * 4))
    pad[:r, :b] = s
    return pad.reshape(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _store(x):
    """A matrix in MXFP4 storage: (codes, scales)."""
    codes, s = _quantize(x)
    return _pack(codes), _tile_scales(s)


def _values(codes, scales, rows, cols):
    """What MXFP4 storage stands for, in fp32."""
    lev = _levels(codes.device)
    v = torch.stack([lev[(codes & 15).int()], lev[(codes >> 4).int()]], 2).reshape(rows, cols // BLOCK, BLOCK)
    rt, bt = -(-rows // 128), -(-(cols // BLOCK) // 4)
    s = scales.reshape(rt, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, bt * 4)[:rows, :cols // BLOCK]
    return torch.ldexp(v, s.int().unsqueeze(2) - 127).reshape(rows, cols)


def _rounded(x):
    """The values of a matrix after MXFP4 quantisation along its rows, in fp32."""
    codes, s = _quantize(x)
    v = _levels(x.device)[codes.int()].reshape(x.shape[0], -1, BLOCK)
    return torch.ldexp(v, s.int().unsqueeze(2) - 127).reshape(x.shape)


# --------------------------------------------------- plain form: generator
def _mulhilo(a, m):
    """High and low 32 bits of a * m, a < 2^32 in int64, m a 32-bit constant."""
    lo, hi = (a & 0xFFFF) * m, (a >> 16) * m
    mid = hi + (lo >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)


def _keep(n, p, seed, offset, device):
    """Which of n elements dropout keeps: element i takes 16 bits of Philox4x32-10 with key `seed` and counter
    (i / 8, offset) and is kept where they are at least round(65536 p)."""
    q = torch.arange(-(-n // 8), dtype=torch.int64, device=device)
    c = [q & 0xFFFFFFFF, q >> 32, torch.full_like(q, offset & 0xFFFFFFFF), torch.full_like(q, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(c[0], 0xD2511F53)
        h1, l1 = _mulhilo(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    bits = torch.stack([w for x in c for w in (x & 0xFFFF, x >> 16)], 1).reshape(-1)[:n]
    return bits >= round(65536 * p)


def _inv(p):
    return 65536.0 / (65536 - round(65536 * p))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, cols, g):
    """Normal activations with a few outlier channels, as transformer blocks have them."""
    big = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.005, 16.0, 1.0)
    return torch.randn((rows, cols), generator=g, device="cuda") * big


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    r64 = lambda: int(torch.randint(0, 1 << 62, (1,), generator=g, device="cuda"))  # noqa: E731
    st = {"case": case}
    if op == "quantize":
        x = _activations(case["rows"], case["cols"], g)
        st["X"] = (x * 0.02 if case["transpose"] else x).to(DTYPES[case["dtype"]])
    elif op == "dropout":
        st["X"] = torch.randn(case["n"], generator=g, device="cuda").to(DTYPES[case["dtype"]])
        st["seed"], st["offset"] = r64(), r64() & 0xFFFF
    else:
        M, N, K = case["M"], case["N"], case["K"]
        W = (torch.randn((N, K), generator=g, device="cuda") * 0.02).bfloat16()
        st["W"] = _store(W)
        if op == "matmul":
            st["X"] = _store(_activations(M, K, g).bfloat16())
        else:
            r = case["r"]
            st["s"] = 16.0 / r
            st["X"] = _activations(M, K, g).bfloat16()
            st["L1"] = (torch.randn((K, r), generator=g, device="cuda") / math.sqrt(K)).bfloat16()
            st["L2"] = (torch.randn((r, N), generator=g, device="cuda") * 0.02).bfloat16()
            st["seed"], st["offset"] = r64(), r64() & 0xFFFF
            if op == "linear_bwd":
                st["WT"] = _store(W.t().contiguous())
                st["dY"] = (torch.randn((M, N), generator=g, device="cuda") * 0.01).bfloat16()
                st["T"] = torch.randn((M, r), generator=g, device="cuda")
    return st


# --------------------------------------------------------------------- run
def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    import bit_nf4_quantized_15_b200 as q

    c = st["case"]
    if c["op"] == "quantize":
        return q.mx_dequant(q.mx_quantize(st["X"], transpose=c["transpose"]))
    if c["op"] == "dropout":
        return q.dropout(st["X"], c["p"], st["seed"], st["offset"])
    M, N, K = c["M"], c["N"], c["K"]
    w = q.MXTensor(*st["W"], N, K)
    if c["op"] == "matmul":
        return q.mx_matmul(q.MXTensor(*st["X"], M, K), w)
    drop = q.Dropout(c["p"], st["seed"], st["offset"]) if c["p"] else None
    if c["op"] == "linear_fwd":
        return q.mx_linear_fwd(st["X"], q.MXWeight(w), st["L1"], st["L2"], st["s"], dropout=drop)
    w = q.MXWeight(w, q.MXTensor(*st["WT"], K, N))
    return q.mx_linear_bwd(st["dY"], st["X"], st["T"], w, st["L1"], st["L2"], st["s"], dropout=drop)


def _plain(st):
    c = st["case"]
    if c["op"] == "quantize":
        x = st["X"].t() if c["transpose"] else st["X"]
        return _rounded(x).bfloat16()
    if c["op"] == "dropout":
        x = st["X"]
        keep = _keep(c["n"], c["p"], st["seed"], st["offset"], x.device)
        return torch.where(keep, x.float() * _inv(c["p"]), 0.0).to(x.dtype)
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "matmul":
        return (_values(*st["X"], M, K) @ _values(*st["W"], N, K).t()).bfloat16()
    X, L1, L2, s = st["X"].float(), st["L1"].float(), st["L2"].float(), st["s"]
    keep = _keep(M * K, c["p"], st["seed"], st["offset"], X.device).reshape(M, K) if c["p"] else None
    drop = lambda v: v if keep is None else torch.where(keep, v * _inv(c["p"]), 0.0)  # noqa: E731
    if c["op"] == "linear_fwd":
        T = drop(X) @ L1
        return (_rounded(X) @ _values(*st["W"], N, K).t() + s * (T @ L2)).bfloat16(), T
    dY = st["dY"].float()
    dT = s * (dY @ L2.t())
    dX = _rounded(dY) @ _values(*st["WT"], K, N).t() + drop(dT @ L1.t())
    return dX.bfloat16(), drop(X).t() @ dT, s * (st["T"].t() @ dY)


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    mx = 0.5 + 1.0 / BLOCK  # bytes an element
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (SIZES[case["dtype"]] + mx + 2), "flops": 2 * n}
    if op == "dropout":
        return {"bytes": 2 * case["n"] * SIZES[case["dtype"]], "flops": 2 * case["n"]}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "matmul":
        return {"bytes": (M + N) * K * mx + 2 * M * N, "flops": 2 * M * N * K}
    r = case["r"]
    adapters = 2 * r * (K + N)
    if op == "linear_fwd":
        return {"bytes": N * K * mx + 2 * M * K + 2 * M * N + 4 * M * r + adapters, "flops": 2 * M * (N * K + r * (N + K))}
    return {"bytes": N * K * mx + 4 * M * K + 2 * M * N + 4 * M * r + 3 * adapters, "flops": 2 * M * (N * K + 2 * r * (N + K))}


# ------------------------------------------------------------------- exact
def _exact_rounded(x):
    """MXFP4 values of a matrix in fp64: the exponent by frexp, the nearest level by distance."""
    b = x.double().reshape(x.shape[0], -1, BLOCK)
    m = b.abs().amax(2, keepdim=True)
    e = torch.where(m > 0, torch.frexp(m)[1] - 3, -127).clamp_min(-127)
    scale = torch.exp2(e.double())
    lev = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    a = b.abs() / scale
    best, dist = torch.zeros_like(a), a.clone()
    odd = False
    for v in lev[1:]:
        odd = not odd
        d = (a - v).abs()
        take = d < dist if odd else d <= dist  # a tie goes to the even code
        best, dist = torch.where(take, v, best), torch.minimum(d, dist)
    return (torch.sign(b) * best * scale).reshape(x.shape)


def _exact_values(codes, scales, rows, cols):
    """MXFP4 storage in fp64, the scale of each element looked up by its index."""
    dev = codes.device
    nib = torch.stack([codes & 15, codes >> 4], 2).reshape(rows, cols).long()
    mag, expo = nib & 1, (nib >> 1) & 3
    val = torch.where(expo > 0, (2 + mag).double() * torch.exp2((expo - 2).double()), mag.double() / 2)
    val = torch.where(nib >= 8, -val, val)
    i = torch.arange(rows, device=dev).unsqueeze(1)
    j = torch.arange(cols // BLOCK, device=dev).unsqueeze(0)
    tile = (i // 128) * ((cols + 127) // 128) + j // 4
    at = tile * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4
    s = torch.exp2(scales.long()[at.reshape(-1)].double() - 127).reshape(rows, -1)
    return (val.reshape(rows, -1, BLOCK) * s.unsqueeze(2)).reshape(rows, cols)


def _exact_keep(n, p, seed, offset, device):
    """The generator once more, its products by halves of the constants."""
    mask = (1 << 32) - 1

    def mul(a, m):
        m0, m1 = m & 0xFFFF, m >> 16
        x, y = a * m0, a * m1
        return (y + (x >> 16)) >> 16, (x + ((y & 0xFFFF) << 16)) & mask

    i = torch.arange((n + 7) // 8, device=device, dtype=torch.int64)
    x0, x1, x2, x3 = i & mask, i >> 32, torch.zeros_like(i) + (offset & mask), torch.zeros_like(i) + (offset >> 32)
    for rnd in range(10):
        k0 = ((seed & mask) + rnd * 0x9E3779B9) & mask
        k1 = ((seed >> 32) + rnd * 0xBB67AE85) & mask
        a1, a0 = mul(x0, 0xD2511F53)
        b1, b0 = mul(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = b1 ^ x1 ^ k0, b0, a1 ^ x3 ^ k1, a0
    words = torch.stack((x0, x1, x2, x3), 1).unsqueeze(2)
    halves = torch.cat((words & 0xFFFF, words >> 16), 2).reshape(-1)
    return halves[:n] >= int(p * 65536 + 0.5)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_rounded(st["X"].t().contiguous() if case["transpose"] else st["X"])
    if op == "dropout":
        keep = _exact_keep(case["n"], case["p"], st["seed"], st["offset"], "cuda")
        return st["X"].double() * keep / (1 - int(case["p"] * 65536 + 0.5) / 65536)
    M, N, K = case["M"], case["N"], case["K"]
    if op == "matmul":
        return _exact_values(*st["X"], M, K) @ _exact_values(*st["W"], N, K).t()
    X, L1, L2, s = st["X"].double(), st["L1"].double(), st["L2"].double(), st["s"]
    m = 1.0
    if case["p"]:
        m = _exact_keep(M * K, case["p"], st["seed"], st["offset"], "cuda").reshape(M, K).double()
        m = m / (1 - int(case["p"] * 65536 + 0.5) / 65536)
    if op == "linear_fwd":
        T = (X * m) @ L1
        return _exact_rounded(st["X"]) @ _exact_values(*st["W"], N, K).t() + (T * s) @ L2, T
    dY = st["dY"].double()
    dT = dY @ L2.t()
    dX = _exact_rounded(st["dY"]) @ _exact_values(*st["WT"], K, N).t() + ((dT @ L1.t()) * m) * s
    return dX, ((X * m).t() @ dT) * s, (st["T"].double().t() @ dY) * s
