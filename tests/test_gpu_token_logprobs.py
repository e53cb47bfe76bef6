"""sts_token_logprobs and its gradient against the definitions in float64 (numpy, CPU).

Tolerances, with u = 2^-24 (half a step of fp32). A thread of the kernel sums n = V / 256 + 40
terms (its share, and the joins), each an exponential of the hardware (2 u relative, at most 8 u
with its flush) of an argument with three roundings, so a sum is within (n + 64) u relative where
the terms that matter have arguments within 20 (their error 3 u * 20 is part of the 64); that is
the absolute error of its logarithm. Values add a rounding each: 4 u times their size.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def _rows(seed, T, V, dtype, pad=0, mask=None, scale=2.0):
    gen = torch.Generator().manual_seed(seed)
    z = torch.randn(T, V + pad, generator=gen) * scale
    hot = torch.randint(V, (T, 4), generator=gen)
    z.scatter_add_(1, hot, 6.0 * torch.rand(T, 4, generator=gen))
    if mask is not None:
        z[torch.rand(T, V + pad, generator=gen) < 0.4] = -np.inf if mask == "inf" else torch.finfo(DTYPES[dtype]).min
    z = z.to(DTYPES[dtype])
    tau = torch.rand(T, generator=gen) + 0.5
    return z, tau, gen


def _tokens(gen, T, V, m):
    y = torch.randint(V, (T, m), generator=gen)
    if m >= 3:
        y[:, 1] = y[:, 0]  # the same token twice
        y[::2, 2] = -1
    return y


def reference(z, tau, tokens, n):
    """Definitions in float64, row by row; z float64 (exactly the logits)."""
    T, V = z.shape
    out = dict(logprob=np.zeros(tokens.shape), entropy=np.zeros(T), lse=np.zeros(T), mean_d=np.zeros(T),
               top_id=np.full((T, n), -1, np.int64), top_logprob=np.full((T, n), -np.inf), p=np.zeros((T, V)),
               lp=np.full((T, V), -np.inf))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        for t in range(T):
            zmax = z[t].max()
            if zmax == -np.inf:
                out["logprob"][t] = np.where(tokens[t] < 0, 0.0, -np.inf)
                out["lse"][t] = -np.inf
                continue
            d = (z[t] - zmax) / tau[t]
            e = np.exp(d)
            S = e.sum()
            out["lse"][t] = zmax / tau[t] + np.log(S)
            lp = d - np.log(S)
            p = e / S
            kept = p > 0
            out["mean_d"][t] = -(p[kept] * d[kept]).sum()
            out["entropy"][t] = -(p[kept] * lp[kept]).sum()
            out["logprob"][t] = np.where(tokens[t] < 0, 0.0, lp[np.maximum(tokens[t], 0)])
            order = np.lexsort((np.arange(V), -(z[t] + 0.0)))[:n]
            order = order[z[t][order] > -np.inf]
            out["top_id"][t, :len(order)] = order
            out["top_logprob"][t, :len(order)] = lp[order]
            out["p"][t], out["lp"][t] = p, lp
    return out


def _f32_overflow(lp):
    """A logprob beyond fp32's range (its largest value, 2^128 - 2^104, and half a step) is -inf there."""
    return np.where(lp <= -(2.0 ** 128 - 2.0 ** 103), -np.inf, lp)


def _close(got, want, tol):
    got, want = got.double().cpu().numpy(), _f32_overflow(want)
    fin = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fin)
    assert np.array_equal(got[~fin], want[~fin])
    with np.errstate(invalid="ignore"):  # equal infinities
        err = np.abs(got - want)[fin]
    tol = np.broadcast_to(tol, want.shape)[fin]
    assert (err <= tol).all(), f"max error {err.max()} at tolerance {tol[err.argmax()]}"


def _check_forward(z, tau, tokens, n, got, saved, V):
    ref = reference(z.double().cpu().numpy(), tau.double().cpu().numpy(), tokens.cpu().numpy(), n)
    sum_tol = (V / 256 + 40 + 64) * U
    tol = lambda v: sum_tol + 4 * U * np.where(np.isfinite(v), np.abs(v), 0.0)  # noqa: E731
    _close(got, ref["logprob"], tol(ref["logprob"]))
    if n:
        assert np.array_equal(saved["top_id"].cpu().numpy(), ref["top_id"])
        _close(saved["top_logprob"], ref["top_logprob"], tol(ref["top_logprob"]))
    _close(saved["lse"], ref["lse"], tol(ref["lse"]))
    _close(saved["entropy"], ref["entropy"], sum_tol * (2 + ref["mean_d"]) + 4 * U * ref["entropy"])
    return ref


CASES = [  # T, V, m, n, dtype, pad, mask
    (1, 1, 1, 1, "fp32", 0, None),
    (3, 2, 3, 5, "bf16", 0, None),
    (5, 7, 1, 0, "fp16", 1, None),
    (2, 8, 4, 8, "bf16", 8, None),
    (4, 33, 2, 64, "fp32", 3, "inf"),
    (700, 257, 3, 20, "fp32", 1, "inf"),
    (640, 1000, 8, 64, "fp16", 0, "lowest"),
    (9, 4097, 64, 20, "bf16", 1, None),
    (17, 8191, 1, 64, "fp32", 0, "lowest"),
    (600, 8200, 1, 1, "bf16", 0, None),
    (1, 50021, 512, 64, "fp16", 0, "inf"),
    (3, 151936, 1, 20, "fp32", 0, None),
    (600, 20003, 2, 8, "bf16", 5, "lowest"),
    (2, 262144, 5, 64, "bf16", 0, None),
]


@pytest.mark.parametrize("T,V,m,n,dtype,pad,mask", CASES)
def test_forward_matches_the_definition(cuda_lib, T, V, m, n, dtype, pad, mask):
    z, tau, gen = _rows(T * 7 + V, T, V, dtype, pad, mask)
    tokens = _tokens(gen, T, V, m)
    if mask == "inf" and T > 1:
        z[T // 2] = -np.inf
    held = z.cuda()
    view = held[:, :V]
    lp, saved = cuda_lib.sts_token_logprobs(view, tokens.cuda(), temperature=tau.cuda(), top_n=n, entropy=True)
    _check_forward(z[:, :V], tau, tokens, n, lp, saved, V)
    assert torch.equal(held.cpu(), z)  # the logits are left alone


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("off", [1, 3, 5])
def test_rows_off_any_vector_boundary(cuda_lib, dtype, off):
    V = 3001
    z, tau, gen = _rows(off, 6, V + off, dtype)
    tokens = _tokens(gen, 6, V, 2)
    lp, saved = cuda_lib.sts_token_logprobs(z.cuda()[:, off:], tokens.cuda(), temperature=tau.cuda(), top_n=7, entropy=True)
    _check_forward(z[:, off:], tau, tokens, 7, lp, saved, V)


def _hard_rows(V, dtype):
    """Rows that the order of the vocabulary or the masks make awkward."""
    lowest = torch.finfo(DTYPES[dtype]).min
    i = torch.arange(V, dtype=torch.float64)
    rows = {
        "constant": torch.zeros(V, dtype=torch.float64),
        "ascending": i / V * 8,
        "descending": -i / V * 8,
        "two values": (i % 2) * 3,
        "steps": torch.floor(i / 100),
        "signed zeros": torch.where(i % 3 == 0, -0.0, 0.0).double(),
        "all lowest": torch.full((V,), lowest, dtype=torch.float64),
        "lowest but one": torch.where(i == V - 1, 1.0, lowest).double(),
        "last only": torch.where(i == V - 1, 2.0, -np.inf).double(),
        "tail only": torch.where(i >= V - 5, i - V, -np.inf).double(),
        "first half masked": torch.where(i < V // 2, -np.inf, torch.sin(i)).double(),
        "far below": -20000.0 + torch.sin(i),
        "far above": 20000.0 + torch.sin(i) * 100,
        "one peak": torch.where(i == V // 3, 60.0, 0.0).double(),
        "rising past the base": torch.where(i > V - 20, 500.0 + 16 * (i - V), torch.cos(i)).double(),
        "nothing": torch.full((V,), -np.inf, dtype=torch.float64),
    }
    return list(rows), torch.stack(list(rows.values())).to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [601, 40000])
@pytest.mark.parametrize("copies", [1, 60])  # clusters of blocks, and one block a row
def test_hard_rows(cuda_lib, dtype, V, copies):
    names, z = _hard_rows(V, dtype)
    z = z.repeat(copies, 1)
    T = z.shape[0]
    gen = torch.Generator().manual_seed(3)
    tau = (torch.rand(T, generator=gen) + 0.5) if copies == 1 else torch.ones(T)
    tokens = torch.randint(V, (T, 3), generator=gen)
    tokens[:, 2] = V - 1
    lp, saved = cuda_lib.sts_token_logprobs(z.cuda(), tokens.cuda(), temperature=tau.cuda(), top_n=40, entropy=True)
    few = slice(0, len(names))  # the copies have the same logits
    _check_forward(z[few], tau[few], tokens[few], 40, lp[few], {k: v[few] for k, v in saved.items()}, V)
    flags = saved["flags"].cpu().reshape(copies, -1)
    assert (flags[:, names.index("nothing")] == cuda_lib.ROW_EMPTY).all()
    assert (flags[:, :names.index("nothing")] == 0).all()
    assert torch.equal(saved["top_id"].reshape(copies, len(names), -1)[-1], saved["top_id"][few])


@pytest.mark.parametrize("T", [2, 700])
def test_logits_that_outgrow_the_first_base(cuda_lib, T):
    """Scaled logits beyond 2^20, from the start or only later, both signs: the sums change their form on the way."""
    V = 30000
    i = torch.arange(V, dtype=torch.float64)
    late = torch.cos(i)
    late[-9:] = 5.0e6 + torch.arange(9).double()  # fp32 holds these
    early = 3.0e6 - torch.floor(i / 3000)
    below = -4.0e6 + (i % 7)
    steps = torch.where(i > 20000, 1.2e6, torch.where(i > 9000, 6.0e5, 0.0)).double() + (i % 5)
    rows = torch.stack([late, early, below, steps]).float()
    z = rows.repeat(-(-T // 4) + 1, 1)[:max(T, 4)]
    tau = torch.full((z.shape[0],), 0.75)
    gen = torch.Generator().manual_seed(1)
    tokens = torch.randint(V, (z.shape[0], 2), generator=gen)
    tokens[:, 1] = V - 1
    lp, saved = cuda_lib.sts_token_logprobs(z.cuda(), tokens.cuda(), temperature=tau.cuda(), top_n=6, entropy=True)
    few = slice(0, 4)
    _check_forward(z[few], tau[few], tokens[few], 6, lp[few], {k: v[few] for k, v in saved.items()}, V)
    assert torch.equal(saved["entropy"][-4:].sort().values, saved["entropy"][few].sort().values) or z.shape[0] % 4
    g = torch.ones(z.shape[0], 2, device="cuda")
    dz = cuda_lib.sts_token_logprobs_backward(z.cuda(), tokens.cuda(), saved, g, temperature=tau.cuda())
    assert torch.isfinite(dz).all() and dz.double().sum(1).abs().max() < 1e-3  # a gradient of log probabilities sums to 0


def test_invalid_rows_do_not_touch_their_neighbours(cuda_lib):
    sts = cuda_lib
    V = 9000
    for T in (8, 900):  # with and without clusters
        z, tau, gen = _rows(5, T, V, "fp32")
        tokens = torch.randint(V, (T, 2), generator=gen)
        clean = sts.sts_token_logprobs(z.cuda(), tokens.cuda(), temperature=tau.cuda(), top_n=4, entropy=True)
        z[0, 0] = np.nan
        z[1, V - 1] = np.nan
        z[2, 5000] = np.inf
        tau[3] = 0.0
        tau[4] = np.nan
        tokens[5, 1] = V
        tokens[6, 0] = -2
        lp, saved = sts.sts_token_logprobs(z.cuda(), tokens.cuda(), temperature=tau.cuda(), top_n=4, entropy=True)
        bad = sts.ROW_INVALID
        assert saved["flags"][:8].tolist() == [
            bad | sts.ROW_BAD_LOGIT, bad | sts.ROW_BAD_LOGIT, bad | sts.ROW_BAD_LOGIT, bad | sts.ROW_BAD_TEMPERATURE,
            bad | sts.ROW_BAD_TEMPERATURE, bad | sts.ROW_BAD_TARGET, bad | sts.ROW_BAD_TARGET, 0]
        assert torch.isnan(lp[:7]).all() and (saved["top_id"][:7] == -1).all()
        for k in ("lse", "entropy", "logit_max", "log_sum", "top_logprob"):
            assert torch.isnan(saved[k][:7]).all(), k
        assert torch.equal(lp[7:], clean[0][7:])
        for k, v in clean[1].items():
            assert torch.equal(saved[k][7:], v[7:]), k
        dz = sts.sts_token_logprobs_backward(z.cuda(), tokens.cuda(), saved, torch.ones(T, 2, device="cuda"),
                                             grad_entropy=torch.ones(T, device="cuda"), temperature=tau.cuda())
        assert (dz[:7] == 0).all() and torch.isfinite(dz).all()
        with pytest.raises(sts.StsError) as e:
            sts.sts_token_logprobs(z.cuda(), tokens.cuda(), temperature=tau.cuda(), check=True)
        assert "row 0" in str(e.value)


def test_extreme_temperatures(cuda_lib):
    V = 5000
    z, _, gen = _rows(9, 4, V, "fp32")
    tau = torch.tensor([1e-30, 1e-3, 1e4, 1e30])
    tokens = z.argmax(1, keepdim=True)
    lp, saved = cuda_lib.sts_token_logprobs(z.cuda(), tokens.cuda(), temperature=tau.cuda(), top_n=3, entropy=True)
    _check_forward(z, tau, tokens, 3, lp, saved, V)


def _grad_reference(z, tau, tokens, n, g, h, gt, ref):
    T, V = z.shape
    dz = np.zeros((T, V))
    size = np.zeros((T, V))  # the sum of the magnitudes that meet in an element
    for t in range(T):
        if ref["lse"][t] == -np.inf:
            continue
        p, lp = ref["p"][t], np.where(ref["p"][t] > 0, ref["lp"][t], 0.0)
        G = 0.0
        mass = 0.0
        for ids, gs in ((tokens[t], g[t]), (ref["top_id"][t], gt[t] if gt is not None else [])):
            for y, gy in zip(ids, gs):
                if y >= 0 and z[t, y] > -np.inf:
                    dz[t, y] += gy
                    size[t, y] += abs(gy)
                    G += gy
                    mass += abs(gy)
        hh = 0.0 if h is None else h[t]
        dz[t] -= p * (G + hh * (lp + ref["entropy"][t]))
        # relative error of p: its exponent's roundings, and the saved log_sum's
        rel = (V / 256 + 40 + 64 + 16) * U + 4 * U * np.abs(lp)
        size[t] = 4 * U * size[t] + p * (mass + abs(hh) * (np.abs(lp) + ref["entropy"][t])) * rel
        size[t] += p * abs(hh) * (V / 256 + 104) * U * (2 + ref["mean_d"][t])  # the saved entropy's error
    return dz / tau[:, None], size / tau[:, None]


@pytest.mark.parametrize("T,V,m,n,dtype,pad,mask", CASES)
def test_gradient_matches_the_formula(cuda_lib, T, V, m, n, dtype, pad, mask):
    sts = cuda_lib
    z, tau, gen = _rows(T * 11 + V, T, V, dtype, pad, mask)
    if mask == "inf" and T > 1:
        z[T // 2] = -np.inf
    tokens = _tokens(gen, T, V, m)
    g = torch.randn(T, m, generator=gen)
    h = torch.randn(T, generator=gen)
    gt = torch.randn(T, n, generator=gen) if n else None
    view = z.cuda()[:, :V]
    _, saved = sts.sts_token_logprobs(view, tokens.cuda(), temperature=tau.cuda(), top_n=n, entropy=True)
    dz = sts.sts_token_logprobs_backward(view, tokens.cuda(), saved, g.cuda(), grad_entropy=h.cuda(),
                                         grad_top=None if gt is None else gt.cuda(), temperature=tau.cuda())
    assert dz.dtype == DTYPES[dtype] and dz.shape == (T, V)
    z64, tau64 = z[:, :V].double().numpy(), tau.double().numpy()
    ref = reference(z64, tau64, tokens.numpy(), n)
    want, tol = _grad_reference(z64, tau64, tokens.numpy(), n, g.double().numpy(), h.double().numpy(),
                                None if gt is None else gt.double().numpy(), ref)
    tiny = {"fp32": 1e-37, "bf16": 1e-37, "fp16": 2.0 ** -24}[dtype]  # flushed or subnormal results
    err = np.abs(dz.double().cpu().numpy() - want)
    lim = tol + HALF_STEP[dtype] * (np.abs(want) + tol) + tiny
    assert (err <= lim).all(), (err / lim).max()


@pytest.mark.parametrize("src", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("dst", ["fp32", "bf16", "fp16"])
def test_gradient_types_strides_and_place(cuda_lib, src, dst):
    """Any type to any type, into a strided output whose padding is left alone; in place where the types agree."""
    sts = cuda_lib
    T, V, m = 5, 4099, 4
    z, tau, gen = _rows(2, T, V, src)
    tokens = _tokens(gen, T, V, m).cuda()
    g = torch.randn(T, m, generator=gen).cuda()
    z, tau = z.cuda(), tau.cuda()
    _, saved = sts.sts_token_logprobs(z, tokens, temperature=tau)
    plain = sts.sts_token_logprobs_backward(z, tokens, saved, g, temperature=tau, out_dtype=torch.float32)
    held = torch.full((T, V + 5), 7.0, dtype=DTYPES[dst], device="cuda")
    out = sts.sts_token_logprobs_backward(z, tokens, saved, g, temperature=tau, out=held[:, 1:V + 1])
    assert torch.equal(out, plain.to(DTYPES[dst]))
    assert (held[:, 0] == 7).all() and (held[:, V + 1:] == 7).all()
    if src == dst:
        for rows in (slice(0, T), slice(0, 1)):
            buf = z[rows].clone()
            sv = {k: v[rows] for k, v in saved.items()}
            got = sts.sts_token_logprobs_backward(buf, tokens[rows], sv, g[rows], temperature=tau[rows], out=buf)
            assert got is buf and torch.equal(buf, plain[rows].to(DTYPES[dst]))


def test_gradient_against_differences(cuda_lib):
    """Central differences of the float64 definition (step 1e-4: error about 1e-8 plus the kernel's 1e-6)."""
    sts = cuda_lib
    T, V, n = 3, 9, 2
    z, tau, gen = _rows(4, T, V, "fp32")
    tokens = torch.tensor([[0, 3, 3], [8, -1, 2], [5, 5, 5]])
    g = torch.randn(T, 3, generator=gen)
    h = torch.randn(T, generator=gen)
    gt = torch.randn(T, n, generator=gen)
    _, saved = sts.sts_token_logprobs(z.cuda(), tokens.cuda(), temperature=tau.cuda(), top_n=n, entropy=True)
    dz = sts.sts_token_logprobs_backward(z.cuda(), tokens.cuda(), saved, g.cuda(), grad_entropy=h.cuda(), grad_top=gt.cuda(),
                                         temperature=tau.cuda()).double().cpu().numpy()

    def loss(x):
        r = reference(x, tau.double().numpy(), tokens.numpy(), n)
        return float((r["logprob"] * g.double().numpy()).sum() + (r["entropy"] * h.double().numpy()).sum()
                     + (r["top_logprob"] * gt.double().numpy()).sum())

    x = z.double().numpy()
    for t in range(T):
        for i in range(V):
            up, down = x.copy(), x.copy()
            up[t, i] += 1e-4
            down[t, i] -= 1e-4
            assert abs((loss(up) - loss(down)) / 2e-4 - dz[t, i]) < 1e-5


def test_parts_of_the_gradient_alone(cuda_lib):
    """Each upstream gradient may be left out; without any the result is zero."""
    sts = cuda_lib
    T, V = 4, 3000
    z, tau, gen = _rows(6, T, V, "fp32")
    z, tau = z.cuda(), tau.cuda()
    tokens = torch.randint(V, (T,), generator=gen).cuda()  # [T]: one token a row
    lp, saved = sts.sts_token_logprobs(z, tokens, temperature=tau, top_n=3, entropy=True)
    assert lp.shape == (T,)
    g, h, gt = (torch.randn(s, generator=gen).cuda() for s in ((T,), (T,), (T, 3)))
    call = lambda **k: sts.sts_token_logprobs_backward(z, tokens, saved, temperature=tau, **k)  # noqa: E731
    whole = call(grad_logprob=g, grad_entropy=h, grad_top=gt)
    parts = call(grad_logprob=g) + call(grad_entropy=h) + call(grad_top=gt)
    assert torch.allclose(whole, parts, rtol=1e-4, atol=1e-5)
    assert (call() == 0).all()
    alone, only = sts.sts_token_logprobs(z, None, temperature=tau, top_n=3)
    assert alone is None and torch.equal(only["top_id"], saved["top_id"])


def test_repeats_streams_and_graphs(cuda_lib):
    """The same results twice, on another stream, and from a captured graph replayed on new data."""
    sts = cuda_lib
    T, V, m, n = 3, 40000, 4, 20
    z, tau, gen = _rows(8, T, V, "bf16")
    z, tau, tokens = z.cuda(), tau.cuda(), _tokens(gen, T, V, m).cuda()
    g = torch.randn(T, m, generator=gen).cuda()

    def both(x, stream=None):
        lp, s = sts.sts_token_logprobs(x, tokens, temperature=tau, top_n=n, entropy=True, stream=stream)
        return lp, s["top_id"], s["entropy"], sts.sts_token_logprobs_backward(x, tokens, s, g, temperature=tau, stream=stream)

    first = both(z)
    for a, b in zip(first, both(z)):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(z, side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    buf = z.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(buf)
    fresh = z.roll(1, 0).contiguous()
    buf.copy_(fresh)
    graph.replay()
    for a, b in zip(held, both(fresh)):
        assert torch.equal(a, b)


def test_far_offsets(cuda_lib):
    """Rows beyond 2^31 elements: the same results as on their own."""
    sts = cuda_lib
    T, V = 15000, 152064
    z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    z[-700:] = (torch.randn(700, V, device="cuda") * 3).bfloat16()
    tokens = torch.randint(V, (T, 2), device="cuda")
    lp, saved = sts.sts_token_logprobs(z, tokens, top_n=5, entropy=True)
    few, part = sts.sts_token_logprobs(z[-700:], tokens[-700:], top_n=5, entropy=True)
    assert torch.equal(lp[-700:], few)
    for k, v in part.items():
        assert torch.equal(saved[k][-700:], v), k
    g = torch.randn(T, 2, device="cuda")
    want = sts.sts_token_logprobs_backward(z[-700:], tokens[-700:], part, g[-700:])
    assert torch.equal(sts.sts_token_logprobs_backward(z, tokens, saved, g, out=z)[-700:], want)


def test_calls_that_overlap(cuda_lib):
    """Forward and gradient calls on several streams at once, as independent calls."""
    sts = cuda_lib
    T, V = 6, 60000
    streams = [torch.cuda.Stream() for _ in range(3)]
    rows = [_rows(20 + i, T, V, "bf16")[0].cuda() for i in range(3)]
    tokens = torch.randint(V, (T, 2), device="cuda")
    g = torch.randn(T, 2, device="cuda")
    torch.cuda.synchronize()
    got = []
    for z, st in zip(rows, streams):
        lp, s = sts.sts_token_logprobs(z, tokens, top_n=9, entropy=True, stream=st)
        got.append((lp, s, sts.sts_token_logprobs_backward(z, tokens, s, g, stream=st)))
    torch.cuda.synchronize()
    for z, (lp, s, dz) in zip(rows, got):
        lp1, s1 = sts.sts_token_logprobs(z, tokens, top_n=9, entropy=True)
        assert torch.equal(lp, lp1) and torch.equal(s["top_id"], s1["top_id"]) and torch.equal(s["entropy"], s1["entropy"])
        assert torch.equal(dz, sts.sts_token_logprobs_backward(z, tokens, s1, g))


def test_no_rows(cuda_lib):
    z = torch.empty(0, 50, device="cuda")
    lp, saved = cuda_lib.sts_token_logprobs(z, torch.empty(0, 2, dtype=torch.int64, device="cuda"), top_n=2)
    assert lp.shape == (0, 2) and saved["top_id"].shape == (0, 2)
    assert cuda_lib.sts_token_logprobs_backward(z, None, saved).shape == (0, 50)


def _check_gradient(sts, z, tau, tokens, n, view, saved, ref, dtype, seed):
    """The gradient from the same saved scalars, of logprobs, entropy and alternatives together."""
    T, V = z.shape
    gen = torch.Generator().manual_seed(seed)
    g, h, gt = torch.randn(T, tokens.shape[1], generator=gen), torch.randn(T, generator=gen), torch.randn(T, n, generator=gen)
    dz = sts.sts_token_logprobs_backward(view, tokens.cuda(), saved, g.cuda(), grad_entropy=h.cuda(), grad_top=gt.cuda(),
                                         temperature=tau.cuda())
    z64, tau64, h64 = z.double().numpy(), tau.double().numpy(), h.double().numpy()
    want, tol = _grad_reference(z64, tau64, tokens.numpy(), n, g.double().numpy(), h64, gt.double().numpy(), ref)
    tiny = {"fp32": 1e-37, "bf16": 1e-37, "fp16": 2.0 ** -24}[dtype]
    # a probability below 2^-126 is flushed to 0 by the exponential, and with it p (G + h (ln p + entropy)) / tau:
    # at tau = 0.01, ln p = -88, |h| = 3 that is 1.2e-38 * 100 * 264 = 3e-34, beyond what `tiny` holds
    size = np.abs(g.double().numpy()).sum(1) + np.abs(gt.double().numpy()).sum(1)
    lp = np.where(np.isfinite(ref["lp"]), np.abs(ref["lp"]), 0.0)
    flush = 2.0 ** -126 * (size[:, None] + np.abs(h64)[:, None] * (lp + ref["entropy"][:, None])) / tau64[:, None]
    err = np.abs(dz.double().cpu().numpy() - want)
    lim = tol + HALF_STEP[dtype] * (np.abs(want) + tol) + tiny + np.where(ref["p"] < 2.0 ** -125, flush, 0.0)
    bad = np.unravel_index((err / lim).argmax(), err.shape)
    assert (err <= lim).all(), (err[bad], lim[bad], want[bad], ref["p"][bad], ref["lp"][bad])


def _between_rows(V, chunk, n, gen):
    """An ordinary first chunk, more than n logits near 500 in the next two, then logits near 400 and 300: far above
    the first chunk, below the n-th largest. Rows differ in where the 400s start; the last has them only at the end."""
    z = torch.randn(4, V, generator=gen)
    for r in range(4):
        high = chunk + torch.randperm(min(2 * chunk, V - chunk), generator=gen)[:n + 8]
        z[r, high] = 500 + torch.randn(len(high), generator=gen)
        start = min((3, 4, 5, 6)[r] * chunk, V - 600) if r < 3 else V - 600
        at = start + torch.randperm(V - start, generator=gen)[:300]
        z[r, at[:200]] = 400 + torch.randn(200, generator=gen)
        z[r, at[200:]] = 300 + torch.randn(100, generator=gen)
    return z


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,copies", [(50021, 150), (152064, 100), (262144, 1)])  # 128 and 256 threads, and clusters
@pytest.mark.parametrize("n", [2, 8, 20, 64])
def test_logits_between_the_first_chunk_and_the_bound(cuda_lib, dtype, V, copies, n):
    """The bound of the alternatives rises over what the first chunk held; logits between the two enter the sums of
    threads that never met one above the bound."""
    gen = torch.Generator().manual_seed(V + n)
    threads = 128 if V <= 65536 else 256
    z = _between_rows(V, threads * 4 * (4 if dtype == "fp32" else 8), n, gen).to(DTYPES[dtype])
    tau = torch.tensor([1.0, 0.7, 1.3, 1.0])
    tokens = torch.randint(V, (4, 2), generator=gen)
    tokens[:, 1] = z.argmax(1)
    view = z.cuda().repeat(copies, 1)
    lp, saved = cuda_lib.sts_token_logprobs(view, tokens.cuda().repeat(copies, 1), temperature=tau.cuda().repeat(copies), top_n=n,
                                            entropy=True)
    assert (saved["flags"] == 0).all()
    few = {k: v[-4:].contiguous() for k, v in saved.items()}
    ref = _check_forward(z, tau, tokens, n, lp[-4:], few, V)
    for k, v in saved.items():
        assert torch.equal(v.reshape(copies, 4, -1), v[-4:].reshape(1, 4, -1).expand(copies, 4, -1)), k
    _check_gradient(cuda_lib, z, tau, tokens, n, view[-4:], few, ref, dtype, n)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,V", [(3, 262144), (300, 152064), (300, 60000)])
@pytest.mark.parametrize("mask", [-100.0, -1000.0])
@pytest.mark.parametrize("n", [2, 5, 20])
def test_a_finite_mask_that_is_added(cuda_lib, dtype, T, V, mask, n):
    """400 allowed tokens, none in the first part of the vocabulary; what is not allowed is lowered, not removed."""
    gen = torch.Generator().manual_seed(V + n)
    rows = 4
    z = torch.randn(rows, V, generator=gen) * 2 + mask
    for r in range(rows):
        allowed = 10000 + torch.randperm(V - 10000, generator=gen)[:400]
        z[r, allowed] -= mask
    z = z.to(DTYPES[dtype])
    tau = torch.ones(rows)
    tokens = torch.randint(V, (rows, 2), generator=gen)
    tokens[:, 1] = z.argmax(1)
    pick = torch.arange(T) % rows
    view = z.cuda()[pick.cuda()]
    lp, saved = cuda_lib.sts_token_logprobs(view, tokens.cuda()[pick.cuda()], top_n=n, entropy=True)
    rows = min(rows, T)
    few = {k: v[:rows].contiguous() for k, v in saved.items()}
    ref = _check_forward(z[:rows], tau[:rows], tokens[:rows], n, lp[:rows], few, V)
    _check_gradient(cuda_lib, z[:rows], tau[:rows], tokens[:rows], n, view[:rows], few, ref, dtype, n)


@pytest.mark.parametrize("dtype,V", [("bf16", 152064), ("fp32", 152064), ("fp16", 50021)])
@pytest.mark.parametrize("temperature", [0.01, 0.02, 0.05])
@pytest.mark.parametrize("n", [2, 5, 64])
def test_low_temperatures_over_a_whole_vocabulary(cuda_lib, dtype, V, temperature, n):
    """Logits as a model gives them (a few hot tokens), a block a row; 32 of the rows against the definition."""
    gen = torch.Generator().manual_seed(n)
    T, few = 640, 32
    z = torch.randn(few, V, generator=gen) * 2
    hot = torch.randint(V, (few, 40), generator=gen)
    z.scatter_add_(1, hot, 4 + 8 * torch.rand(few, 40, generator=gen))
    z = z.to(DTYPES[dtype])
    tau = torch.full((few,), temperature)
    tokens = hot[:, :2].contiguous()
    view = z.cuda().repeat(T // few, 1)
    lp, saved = cuda_lib.sts_token_logprobs(view, tokens.cuda().repeat(T // few, 1), temperature=tau.cuda().repeat(T // few), top_n=n,
                                            entropy=True)
    assert torch.isfinite(saved["lse"]).all() and torch.isfinite(saved["entropy"]).all()
    part = {k: v[-few:].contiguous() for k, v in saved.items()}
    ref = _check_forward(z, tau, tokens, n, lp[-few:], part, V)
    _check_gradient(cuda_lib, z, tau, tokens, n, view[-few:], part, ref, dtype, n)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("mask", ["inf", "lowest"])
def test_gradients_of_masked_tokens_at_low_temperatures(cuda_lib, dtype, mask):
    """A masked token has a gradient of 0 however small the temperature (its difference from the largest logit, times
    the parts of log2(e) / tau, leaves fp32 from 4e-8 on)."""
    sts = cuda_lib
    taus = torch.logspace(-30, -2, 141).tolist()
    T, V = len(taus), 1003
    z, _, gen = _rows(31, T, V, dtype, mask=mask)
    tau = torch.tensor(taus)
    tokens = torch.stack([z.argmax(1), torch.randint(V, (T,), generator=gen)], 1)
    g, h = torch.randn(T, 2, generator=gen), torch.randn(T, generator=gen)
    _, saved = sts.sts_token_logprobs(z.cuda(), tokens.cuda(), temperature=tau.cuda(), entropy=True, check=True)
    dz = sts.sts_token_logprobs_backward(z.cuda(), tokens.cuda(), saved, g.cuda(), grad_entropy=h.cuda(), temperature=tau.cuda(),
                                         out_dtype=torch.float32)
    z64, tau64 = z.double().numpy(), tau.double().numpy()
    ref = reference(z64, tau64, tokens.numpy(), 0)
    want, tol = _grad_reference(z64, tau64, tokens.numpy(), 0, g.double().numpy(), h.double().numpy(), None, ref)
    # a probability below 2^-126 is flushed: |G| + |h| (|ln p| + entropy) <= 8 + 4 (88 + 7), over tau
    flush = np.where((ref["p"] > 0) & (ref["p"] < 2.0 ** -125), 2.0 ** -126 * 400, 0.0) / tau64[:, None]
    err = np.abs(dz.double().cpu().numpy() - want)
    lim = tol + U * (np.abs(want) + tol) + flush
    bad = ~(err <= lim)
    assert not bad.any(), (np.argwhere(bad)[:3], dz.cpu().numpy()[bad][:3], want[bad][:3], lim[bad][:3])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [9, 5003, 40000])
def test_gradients_at_the_smallest_temperatures(cuda_lib, dtype, V):
    """Temperatures down to the smallest fp32: (G + h (ln p + entropy)) / tau leaves fp32, but a token without
    probability has a gradient of 0 and the others theirs, infinite only where the formula's is beyond fp32."""
    sts = cuda_lib
    taus = [1e-30, 1e-35, 1e-36, 1e-37, 1e-38, 1e-40, 1.5e-45]
    T, n = 3 * len(taus), 2
    gen = torch.Generator().manual_seed(V)
    z = torch.randn(T, V, generator=gen)
    z[::3, 3] = 9.0
    z[1::3, [2, V - 1]] = 9.0  # two equal ones
    z[2::3] = -np.inf
    z[2::3, V // 2] = 1.0
    z = z.to(DTYPES[dtype])
    tau = torch.tensor(taus).repeat_interleave(3)
    tokens = torch.stack([z.argmax(1), torch.randint(V, (T,), generator=gen)], 1)
    g, h, gt = torch.randn(T, 2, generator=gen), torch.randn(T, generator=gen), torch.randn(T, n, generator=gen)
    zc = z.cuda()
    lp, saved = sts.sts_token_logprobs(zc, tokens.cuda(), temperature=tau.cuda(), top_n=n, entropy=True)
    assert (saved["flags"] == 0).all() and not torch.isnan(lp).any()
    ref = reference(z.double().numpy(), tau.double().numpy(), tokens.numpy(), n)
    most = {"fp32": torch.finfo(torch.float32).max, "bf16": torch.finfo(torch.bfloat16).max, "fp16": 65504.0}[dtype]
    for hh, top in ((h, gt), (None, None)):
        dz = sts.sts_token_logprobs_backward(zc, tokens.cuda(), saved, g.cuda(), grad_entropy=None if hh is None else hh.cuda(),
                                             grad_top=None if top is None else top.cuda(), temperature=tau.cuda())
        place = zc.clone()
        sts.sts_token_logprobs_backward(place, tokens.cuda(), saved, g.cuda(), grad_entropy=None if hh is None else hh.cuda(),
                                        grad_top=None if top is None else top.cuda(), temperature=tau.cuda(), out=place)
        got = dz.double().cpu().numpy()
        assert not np.isnan(got).any() and np.array_equal(place.double().cpu().numpy(), got)
        want, tol = _grad_reference(z.double().numpy(), tau.double().numpy(), tokens.numpy(), n, g.double().numpy(),
                                    None if hh is None else hh.double().numpy(), None if top is None else top.double().numpy(), ref)
        lim = tol + HALF_STEP[dtype] * (np.abs(want) + tol)
        inside = np.abs(want) + lim < most
        with np.errstate(invalid="ignore"):
            bad = inside & ~(np.abs(got - want) <= lim)
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], lim[bad][:5])
        beyond = np.abs(want) - lim > 2 * most
        assert (got[beyond] == np.sign(want[beyond]) * np.inf).all()
