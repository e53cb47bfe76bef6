"""A head kept in 8 bits: sts_block_quantize and sts_block_scaled_product against float64, and the
path they make with the token log probabilities."""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TOP = {E4M3: 448.0, E5M2: 57344.0}
SRC = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _expand(scale, R, K, block_rows):
    return scale.repeat_interleave(block_rows, 0)[:R].repeat_interleave(128, 1)[:, :K]


def quantize_reference(x, block_rows, dtype):
    """The documented formula with the CPU's IEEE fp32 arithmetic and 8-bit conversion."""
    R, K = x.shape
    x = x.float().cpu()
    Rb, Kb = -(-R // block_rows), -(-K // 128)
    pad = torch.zeros(Rb * block_rows, Kb * 128)
    pad[:R, :K] = x
    b = pad.reshape(Rb, block_rows, Kb, 128)
    finite = torch.isfinite(b)
    scale = torch.where(finite, b.abs(), 0.0).amax((1, 3)) / TOP[dtype]
    scale = torch.where(scale > 0, scale, 1.0)
    s = scale[:, None, :, None]
    y = torch.where(s >= 2.0 ** -126, b * (1.0 / s), b / s)
    q = torch.where(finite, y.clamp(-TOP[dtype], TOP[dtype]), math.nan)
    return q.reshape(Rb * block_rows, Kb * 128)[:R, :K].to(dtype), scale


def _same_codes(got, want):
    a, b = got.float().cpu(), want.float()
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.mark.parametrize("src", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 128), (3, 130), (129, 257), (128, 4096), (300, 1001), (1000, 64)])
def test_quantize(cuda_lib, src, dtype, block_rows, transposed, R, K):
    gen = torch.Generator().manual_seed(R * K)
    shape = (K, R) if transposed else (R, K)
    x = torch.randn(shape, generator=gen) * torch.exp(2 * torch.randn(shape[0], 1, generator=gen))
    x[torch.rand(shape, generator=gen) < 0.05] = 0.0
    x = x.to(SRC[src])
    x = x.t() if transposed else x
    q, scale = cuda_lib.sts_block_quantize(x.cuda(), block_rows=block_rows, dtype=dtype)
    want_q, want_s = quantize_reference(x, block_rows, dtype)
    assert q.shape == (R, K) and q.dtype == dtype and (R == 1 or q.stride(0) % 16 == 0)
    assert torch.equal(scale.cpu(), want_s)
    _same_codes(q, want_q)
    # within half a step of the 8-bit type, and the roundings of the scale and the quotient
    mant, low = (3, -6) if dtype == E4M3 else (2, -14)
    s = _expand(scale.double().cpu(), R, K, block_rows)
    err = (q.double().cpu() * s - x.double()).abs()
    half = torch.maximum(x.double().abs() * 2.0 ** -(mant + 1), s * 2.0 ** (low - mant - 1))
    assert (err <= half * (1 + 8 * U) + 4 * U * x.double().abs()).all()


def test_quantize_layouts(cuda_lib):
    """Odd strides and bases, caller's outputs with padding, other streams, repeats."""
    gen = torch.Generator().manual_seed(1)
    held = torch.randn(40, 515, generator=gen).bfloat16().cuda()
    for view in (held[:, 1:502], held[3:, 5:], held.t()[2:, 3:39], held[::2, :500], held[:1, ::3].t(), held[:, :1]):
        if view.stride(0) != 1 and view.stride(1) != 1 and view.shape[1] != 1:
            continue
        for block_rows in (1, 128):
            want_q, want_s = quantize_reference(view, block_rows, E4M3)
            q, s = cuda_lib.sts_block_quantize(view, block_rows=block_rows)
            assert torch.equal(s.cpu(), want_s)
            _same_codes(q, want_q)
    x = held[:, :300]
    q = torch.full((40, 331), 9, dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.full((40, 7), -1.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cuda_lib.sts_block_quantize(x, q=q[:, 3:303], scale=s[:, 2:5], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want_q, want_s = quantize_reference(x, 1, E4M3)
    _same_codes(q[:, 3:303], want_q)
    assert torch.equal(s[:, 2:5].cpu(), want_s)
    raw = q.view(torch.uint8)
    assert (raw[:, :3] == 9).all() and (raw[:, 303:] == 9).all() and (s[:, :2] == -1).all() and (s[:, 5:] == -1).all()


def test_quantize_refuses_broadcast_views_and_takes_no_rows(cuda_lib):
    one = torch.ones(4, 1, device="cuda")
    for view in (one[:1].expand(5, 1), torch.ones(1, 4, device="cuda").expand(5, 4), one.expand(4, 5)):
        with pytest.raises(cuda_lib.StsError):
            cuda_lib.sts_block_quantize(view)
    q, s = cuda_lib.sts_block_quantize(torch.empty(0, 200, device="cuda"))
    assert q.shape == (0, 200) and s.shape == (0, 2)


def test_quantize_values_at_the_edges(cuda_lib):
    """Zero blocks, NaN and infinities, subnormals, the largest finite values, exact ties."""
    x = torch.zeros(9, 256)
    x[1, 3] = math.nan
    x[1, 4] = 2.0
    x[2, 5], x[2, 6], x[2, 7] = math.inf, -math.inf, -3.0
    x[3] = math.nan
    x[4, :128] = torch.arange(128) * 2.0 ** -149
    x[5, 0], x[5, 1] = torch.finfo(torch.float32).max, 1.0
    x[6, :128] = torch.linspace(-448, 448, 128)
    x[7, :6] = torch.tensor([448.0, 17.0, 19.0, 21.0, -17.0, 2.0 ** -10])  # ties at scale 1
    x[8, 0] = 1e-44
    for dtype in (E4M3, E5M2):
        for src in (x, x.t().contiguous().t()):
            q, s = cuda_lib.sts_block_quantize(src.cuda(), dtype=dtype)
            want_q, want_s = quantize_reference(x, 1, dtype)
            assert torch.equal(s.cpu(), want_s)
            _same_codes(q, want_q)
    q, s = cuda_lib.sts_block_quantize(x.cuda())
    assert s[0].tolist() == [1.0, 1.0] and q[7, :6].float().tolist() == [448.0, 16.0, 20.0, 20.0, -16.0, 0.0]
    assert torch.isnan(q[2, 5:7].float()).all() and q[2, 7].float().item() == -448.0


def _operand(gen, R, K, dtype, block_rows):
    x = torch.randn(R, K, generator=gen)
    q, scale = quantize_reference(x, block_rows, dtype)
    held = torch.zeros(R, -(-K // 16) * 16, dtype=torch.uint8).view(dtype)
    held.view(torch.uint8)[:, :K] = q.view(torch.uint8)
    return held.cuda()[:, :K], scale.cuda()


def _product_reference(A, sa, B, sb, b_rows, tau=None):
    """float64, and the sum of the magnitudes that enter each element."""
    M, K = A.shape
    a = A.double() * _expand(sa.double(), M, K, 1)
    b = B.double() * _expand(sb.double(), B.shape[0], K, b_rows)
    C, size = a @ b.t(), a.abs() @ b.abs().t()
    if tau is not None:
        C, size = C / tau.double()[:, None], size / tau.double()[:, None]
    return C, size


def _product_tol(C, size, K, out):
    """A block's 128 products are exact; their sum takes at most 128 roundings or truncations of 2 u of what
    is summed; scaling and adding the blocks 2 and one more each; the division and a bf16 result theirs."""
    kb = -(-K // 128)
    tol = size * (128 * 2 * U + (kb + 4) * U)
    return tol + (2.0 ** -8 * (C.abs() + tol) if out == torch.bfloat16 else 0.0)


PRODUCTS = [  # M, N, K, a, b, b_rows, out, tau
    (1, 1, 1, E4M3, E4M3, 1, "fp32", False),
    (1, 127, 16, E4M3, E4M3, 128, "fp32", True),
    (1, 128, 128, E4M3, E4M3, 128, "bf16", False),
    (5, 300, 129, E4M3, E4M3, 1, "fp32", True),
    (16, 1000, 1024, E5M2, E4M3, 128, "fp32", False),
    (17, 129, 4001, E4M3, E4M3, 128, "bf16", True),  # a cluster of 8 per tile
    (33, 257, 2048, E4M3, E5M2, 1, "fp32", False),
    (64, 2048, 4096, E4M3, E4M3, 128, "fp32", True),
    (77, 30011, 640, E4M3, E4M3, 128, "bf16", True),
    (100, 1027, 777, E5M2, E5M2, 1, "fp32", False),
    (70, 21000, 700, E4M3, E4M3, 128, "fp32", True),  # 65 to 128 rows: the wide form
    (90, 300, 4000, E4M3, E4M3, 128, "bf16", True),  # and the narrow one, split over k
    (128, 5000, 129, E5M2, E4M3, 1, "fp32", False),
    (129, 1024, 1025, E4M3, E4M3, 128, "fp32", True),
    (200, 300, 9000, E4M3, E4M3, 1, "bf16", True),  # wide, split over k
    (256, 4000, 300, E4M3, E4M3, 1, "bf16", False),
    (1000, 777, 2047, E5M2, E4M3, 1, "fp32", True),
    (4500, 1500, 512, E4M3, E4M3, 128, "fp32", False),  # more than one raster group
    (3, 152064, 5120, E4M3, E4M3, 128, "fp32", True),
]


@pytest.mark.parametrize("M,N,K,a,b,b_rows,out,tau", PRODUCTS)
def test_product(cuda_lib, M, N, K, a, b, b_rows, out, tau):
    gen = torch.Generator().manual_seed(M + N + K)
    A, sa = _operand(gen, M, K, a, 1)
    B, sb = _operand(gen, N, K, b, b_rows)
    temperature = (torch.rand(M, generator=gen) + 0.5).cuda() if tau else None
    C = cuda_lib.sts_block_scaled_product(A, sa, B, sb, temperature=temperature, out_dtype=SRC[out], check=True)
    want, size = _product_reference(A, sa, B, sb, b_rows, temperature)
    assert C.shape == (M, N) and C.dtype == SRC[out]
    err = (C.double() - want).abs()
    lim = _product_tol(want, size, K, SRC[out])
    assert (err <= lim).all(), float((err / lim).max())
    again = cuda_lib.sts_block_scaled_product(A, sa, B, sb, temperature=temperature, out_dtype=SRC[out])
    assert torch.equal(again, C)


@pytest.mark.parametrize("M,N,K", [(40, 500, 1000), (300, 3000, 200)])
def test_product_strides_accumulation_and_neighbours(cuda_lib, M, N, K):
    """Strided operands, scales and results: only C[:M, :N] is written, with and without adding."""
    gen = torch.Generator().manual_seed(3)
    A, sa = _operand(gen, M, K, E4M3, 1)
    B, sb = _operand(gen, N, K, E4M3, 128)
    plain = cuda_lib.sts_block_scaled_product(A, sa, B, sb)
    wide = torch.zeros(M, 4096, dtype=torch.uint8, device="cuda").fill_(0x7F).view(E4M3)  # NaN around it
    wide.view(torch.uint8)[:, 16:16 + K] = A.view(torch.uint8)
    sa_t = sa.t().contiguous().t()  # block-major scales
    sb_w = torch.full((sb.shape[0], sb.shape[1] * 2), math.nan, device="cuda")
    sb_w[:, ::2] = sb
    held = torch.full((M + 2, N + 3), 5.0, device="cuda")
    out = held[1:-1, 1:N + 1]
    got = cuda_lib.sts_block_scaled_product(wide[:, 16:16 + K], sa_t, B, sb_w[:, ::2], out=out)
    assert got is out and torch.equal(out, plain)
    cuda_lib.sts_block_scaled_product(A, sa, B, sb, out=out, accumulate=True)
    assert torch.equal(out, plain + plain)
    rest = held.clone()
    rest[1:-1, 1:N + 1] = 5.0
    assert (rest == 5.0).all()


@pytest.mark.parametrize("M", [1, 300])
@pytest.mark.parametrize("tiles", [1, 15, 16, 17, 18, 19, 33, 34, 37, 38, 74, 75])
def test_product_around_the_clusters_that_the_device_holds(cuda_lib, M, tiles):
    """Few tiles and a long k: from 8 parts a tile to none, in both forms (16 rows of B a tile, or 128 x 256)."""
    N, K = (tiles * 16, 4200) if M == 1 else (max(1, tiles // 3) * 256, 4200)
    gen = torch.Generator().manual_seed(tiles)
    A, sa = _operand(gen, M, K, E4M3, 1)
    B, sb = _operand(gen, N, K, E4M3, 128)
    C = cuda_lib.sts_block_scaled_product(A, sa, B, sb, check=True)
    want, size = _product_reference(A, sa, B, sb, 128)
    assert ((C.double() - want).abs() <= _product_tol(want, size, K, torch.float32)).all()
    assert torch.equal(C, cuda_lib.sts_block_scaled_product(A, sa, B, sb))


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N", [(300, 739), (129, 3), (1000, 2049), (700, 5003), (40, 501), (300, 256), (200, 777)])
@pytest.mark.parametrize("K", [130, 9000])  # whole, and split over k where there are few tiles
@pytest.mark.parametrize("more", [1, 2, 5, 8])
def test_product_leaves_what_lies_behind_a_row(cuda_lib, out, M, N, K, more):
    """Rows of C that start on 16-byte boundaries and end anywhere: the bytes up to the next row keep their values."""
    gen = torch.Generator().manual_seed(N)
    A, sa = _operand(gen, M, K, E4M3, 1)
    B, sb = _operand(gen, N, K, E4M3, 128)
    ld = -(-(N + more) // 8) * 8
    plain = cuda_lib.sts_block_scaled_product(A, sa, B, sb, out_dtype=SRC[out])
    want, size = _product_reference(A, sa, B, sb, 128)
    assert ((plain.double() - want).abs() <= _product_tol(want, size, K, SRC[out])).all()
    for accumulate in (False, True) if out == "fp32" else (False,):
        held = torch.full((M + 1, ld), -3.0, dtype=SRC[out], device="cuda")
        got = held[:M, :N]
        if accumulate:
            got.zero_()
        cuda_lib.sts_block_scaled_product(A, sa, B, sb, out=got, accumulate=accumulate)
        assert torch.equal(got, plain)
        assert (held[:M, N:] == -3).all() and (held[M] == -3).all()


@pytest.mark.parametrize("M,N,K", [(40, 300, 9000), (300, 400, 9000)])
def test_product_split_over_k_accumulates_and_fits_any_rows(cuda_lib, M, N, K):
    """A cluster per tile, both forms: C off any alignment, added to, its neighbours left alone."""
    gen = torch.Generator().manual_seed(9)
    A, sa = _operand(gen, M, K, E4M3, 1)
    B, sb = _operand(gen, N, K, E4M3, 128)
    held = torch.full((M, N + 3), 5.0, device="cuda")
    cuda_lib.sts_block_scaled_product(A, sa, B, sb, out=held[:, 1:N + 1], accumulate=True)
    want, size = _product_reference(A, sa, B, sb, 128)
    err = (held[:, 1:N + 1].double() - 5 - want).abs()
    assert (err <= _product_tol(want, size, K, torch.float32) + 2 * U * (5 + want.abs())).all()
    assert (held[:, 0] == 5).all() and (held[:, N + 1:] == 5).all()


def test_far_offsets(cuda_lib):
    """Elements beyond 2^31, of the source, the codes and the product."""
    R, K = 540000, 4096
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, K, device="cuda").bfloat16()
    for block_rows in (1, 128):
        q, s = cuda_lib.sts_block_quantize(x, block_rows=block_rows)
        want_q, want_s = quantize_reference(x[-96:], block_rows, E4M3)  # 540,000 = 128 * 4218 + 96
        _same_codes(q[-96:], want_q)
        assert torch.equal(s[-want_s.shape[0]:].cpu(), want_s)
    A, sa = cuda_lib.sts_block_quantize(torch.randn(4200, 128, device="cuda"))
    B, sb = q[:, :128].contiguous(), s[:, :1].contiguous()
    C = cuda_lib.sts_block_scaled_product(A, sa, B, sb)
    assert C.numel() > 2 ** 31
    assert torch.equal(C[-5:, -3:], cuda_lib.sts_block_scaled_product(A[-5:], sa[-5:], B, sb)[:, -3:])
    assert (C[-1, :-3] == 0).all() and (C[-1, -3:] != 0).all()


def test_product_not_finite(cuda_lib):
    """A NaN code reaches its own row or column of C and no other."""
    gen = torch.Generator().manual_seed(4)
    A, sa = _operand(gen, 20, 300, E4M3, 1)
    B, sb = _operand(gen, 200, 300, E4M3, 128)
    A.view(torch.uint8)[7, 299] = 0x7F
    B.view(torch.uint8)[130, 0] = 0xFF
    C = cuda_lib.sts_block_scaled_product(A, sa, B, sb)
    nan = torch.zeros(20, 200, dtype=torch.bool, device="cuda")
    nan[7] = True
    nan[:, 130] = True
    assert torch.equal(torch.isnan(C), nan)


@pytest.mark.parametrize("M,N,K,b_rows,out,block", [
    (5, 30000, 300, 128, "fp32", 3),  # narrow: two tiles of the block's are lost
    (100, 30001, 200, 1, "bf16", 147),
    (1000, 20000, 300, 128, "fp32", 0),  # wide, by TMA
    (1000, 20003, 300, 128, "fp32", 7),  # wide, rows that TMA cannot address
    (700, 20000, 130, 1, "bf16", 11),
    (40, 300, 9000, 128, "fp32", 1),  # a part of a split over k: the whole tile depends on it
    (300, 400, 9000, 1, "fp32", 8),
    (300, 400, 9000, 128, "bf16", 7)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_a_product_that_gives_up_does_not_pass_for_one(cuda_lib, M, N, K, b_rows, out, block, accumulate):
    """A block that gives up leaves NaN where its results belong, nothing else changes, and the status says so."""
    if accumulate and out != "fp32":
        accumulate = False
    gen = torch.Generator().manual_seed(12)
    A, sa = _operand(gen, M, K, E4M3, 1)
    B, sb = _operand(gen, N, K, E4M3, b_rows)
    plain = cuda_lib.sts_block_scaled_product(A, sa, B, sb, out=torch.full((M, N), 7.0, dtype=SRC[out], device="cuda"),
                                              accumulate=accumulate, check=True)
    C = torch.full((M, N), 7.0, dtype=SRC[out], device="cuda")
    probe = cuda_lib.load().sts_probe_product_timeout
    probe(block)
    try:
        cuda_lib.sts_block_scaled_product(A, sa, B, sb, out=C, accumulate=accumulate)
        with pytest.raises(cuda_lib.StsError) as e:
            cuda_lib.sts_block_scaled_product(A, sa, B, sb, check=True)
        assert e.value.status == 11
    finally:
        probe(-1)
    lost = torch.isnan(C)
    assert lost.any() and not lost.all()
    assert torch.equal(C[~lost], plain[~lost])
    again = cuda_lib.sts_block_scaled_product(A, sa, B, sb, out=torch.full_like(C, 7.0), accumulate=accumulate, check=True)
    assert torch.equal(again, plain)


def test_product_empty(cuda_lib):
    gen = torch.Generator().manual_seed(4)
    A, sa = _operand(gen, 4, 64, E4M3, 1)
    B, sb = _operand(gen, 8, 64, E4M3, 1)
    assert cuda_lib.sts_block_scaled_product(A[:0], sa[:0], B, sb).shape == (0, 8)
    assert cuda_lib.sts_block_scaled_product(A, sa, B[:0], sb[:0]).shape == (4, 0)


def test_product_streams_and_graphs(cuda_lib):
    gen = torch.Generator().manual_seed(5)
    A, sa = _operand(gen, 20, 2048, E4M3, 1)
    B, sb = _operand(gen, 600, 2048, E4M3, 128)
    plain = cuda_lib.sts_block_scaled_product(A, sa, B, sb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = cuda_lib.sts_block_scaled_product(A, sa, B, sb, stream=side)
    here = cuda_lib.sts_block_scaled_product(A, sa, B, sb)  # two calls at once
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(plain, other) and torch.equal(plain, here)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = cuda_lib.sts_block_scaled_product(A, sa, B, sb)
    A.view(torch.uint8).copy_(A.view(torch.uint8).roll(1, 0).clone())
    graph.replay()
    assert torch.equal(held, cuda_lib.sts_block_scaled_product(A, sa, B, sb))


def test_scoring_and_training_an_8_bit_head(cuda_lib):
    """The operators together, as a user trains through an 8-bit head: quantise, project, score, differentiate,
    quantise the gradient, and form dH and dW with the same product. Each step is held to float64 on what the step
    before it gave."""
    sts = cuda_lib
    T, d, V, n = 300, 256, 5003, 5
    gen = torch.Generator().manual_seed(6)
    H = torch.randn(T, d, generator=gen).bfloat16().cuda()
    W = (torch.randn(V, d, generator=gen) / math.sqrt(d) * 4).bfloat16().cuda()
    tau = (torch.rand(T, generator=gen) + 0.5).cuda()
    hq, hs = sts.sts_block_quantize(H)
    wq, ws = sts.sts_block_quantize(W, block_rows=128)
    z = sts.sts_block_scaled_product(hq, hs, wq, ws)
    want, size = _product_reference(hq, hs, wq, ws, 128)
    assert ((z.double() - want).abs() <= _product_tol(want, size, d, torch.float32)).all()
    # 8-bit operands are within 2^-4 of the bf16 ones, element by element
    full = H.double() @ W.double().t()
    mag = H.double().abs() @ W.double().abs().t()
    assert ((z.double() - full).abs() <= mag * (2 * 2.0 ** -4 + 2.0 ** -8) + 0.02 * mag.mean()).all()

    y = torch.randint(V, (T, 2), generator=gen).cuda()
    lp, saved = sts.sts_token_logprobs(z, y, temperature=tau, top_n=n, entropy=True, check=True)
    ref = torch.log_softmax(z.double() / tau.double()[:, None], 1)
    assert (lp.double() - ref.gather(1, y)).abs().max() < (V / 256 + 104 + 80) * U  # values up to 20
    # the same rows through the support program with nothing filtered: one meaning of logprob and entropy
    off = (torch.zeros(T, dtype=torch.int32, device="cuda"), torch.ones(T, device="cuda"), torch.zeros(T, device="cuda"))
    s = sts.sts_block_scaled_product(hq, hs, wq, ws, temperature=tau)
    lp1, filtered, _ = sts.sts_resolve_logits(s, y[:, 0].contiguous(), tau, *off, entropy=True, check=True)
    assert (lp1 - lp[:, 0]).abs().max() < 2e-5 and (filtered["entropy"] - saved["entropy"]).abs().max() < 2e-5
    assert torch.equal(filtered["support_size"], torch.full_like(filtered["support_size"], V))

    g = torch.randn(T, 2, generator=gen).cuda()
    h = 0.1 * torch.randn(T, generator=gen).cuda()
    gt = torch.randn(T, n, generator=gen).cuda()
    dz = sts.sts_token_logprobs_backward(z, y, saved, g, grad_entropy=h, grad_top=gt, temperature=tau)
    x = z.double().requires_grad_()
    lsm = torch.log_softmax(x / tau.double()[:, None], 1)
    loss = (lsm.gather(1, y) * g).sum() - ((lsm.exp() * lsm).sum(1) * h).sum() + (lsm.gather(1, saved["top_id"]) * gt).sum()
    loss.backward()
    assert (dz.double() - x.grad).norm() < 1e-5 * x.grad.norm()

    # dH = dz . W: the sum runs over the vocabulary, so W is quantised again across its rows' blocks
    gq, gs = sts.sts_block_quantize(dz, dtype=E5M2)
    wtq, wts = sts.sts_block_quantize(W.t(), block_rows=128)
    dH = sts.sts_block_scaled_product(gq, gs, wtq, wts)
    want, size = _product_reference(gq, gs, wtq, wts, 128)
    assert dH.shape == (T, d) and ((dH.double() - want).abs() <= _product_tol(want, size, V, torch.float32)).all()
    # dW = dz^T . H, added to what is there; the sum runs over 300 tokens
    gtq, gts = sts.sts_block_quantize(dz.t(), dtype=E5M2)
    htq, hts = sts.sts_block_quantize(H.t())
    dW = torch.ones(V, d, device="cuda")
    sts.sts_block_scaled_product(gtq, gts, htq, hts, out=dW, accumulate=True)
    want, size = _product_reference(gtq, gts, htq, hts, 1)
    assert ((dW.double() - 1 - want).abs() <= _product_tol(want, size, T, torch.float32) + 2 * U * (1 + want.abs())).all()
    # both within the 8-bit types' steps of the gradients of the bf16 operands (e5m2 2^-3, e4m3 2^-4)
    for got, true in ((dH, x.grad @ W.double()), (dW - 1, x.grad.t() @ H.double())):
        assert (got.double() - true).norm() < (2.0 ** -3 + 2.0 ** -4) * true.norm()
