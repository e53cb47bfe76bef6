"""What is measured of the 8-bit head and of the token log probabilities.

Four operators of the library's training and serving path beside the bf16 core:

  quantize   sts_block_quantize           bf16 / fp16 / fp32 -> 8-bit codes and one fp32 scale per 1 x 128 or 128 x 128 block
  product    sts_block_scaled_product     C = A . B^T of two such matrices (logits of an 8-bit head, and both of its gradients)
  logprobs   sts_token_logprobs           log probabilities of given tokens, with entropy, logsumexp and the top alternatives
  gradient   sts_token_logprobs_backward  d / d logits of those log probabilities, of the entropy and of the alternatives

``own = False`` computes them in elementary torch operations in 32 bits; ``own = True`` makes the library's calls.
"""

import math

import torch

own = False

BLOCK = 128
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
FLOAT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one token's hidden state before an 8-bit head answers it: the smallest call
        dict(name="quantize-one-token", op="quantize", R=1, K=4096, src="bf16", to="e4m3", block_rows=1, transposed=False),
        # a whole head's weight, laid out in 128 x 128 blocks after an update
        dict(name="quantize-head", op="quantize", R=151936, K=4096, src="bf16", to="e4m3", block_rows=128, transposed=False),
        # the logits' gradient read across its rows, as the weight gradient's product needs it; an odd token count
        dict(name="quantize-gradient-t", op="quantize", R=32768, K=4001, src="bf16", to="e5m2", block_rows=1, transposed=True),
        # the logits of one token: serving at batch size one, bound by reading the head once
        dict(name="product-one-token", op="product", M=1, N=151936, K=4096, a="e4m3", b="e4m3", b_rows=128, out="fp32", temperature=False),
        # a ragged batch of decoded tokens over a vocabulary of odd size
        dict(name="product-batch-ragged", op="product", M=77, N=50021, K=2048, a="e4m3", b="e4m3", b_rows=128, out="bf16", temperature=True),
        # a training batch through the largest head
        dict(name="product-training", op="product", M=4096, N=152064, K=5120, a="e4m3", b="e4m3", b_rows=128, out="fp32", temperature=True),
        # the weight gradient of a slice of the head: the sum runs over an odd number of tokens, both sides in 1 x 128 blocks
        dict(name="product-weight-gradient", op="product", M=32768, N=2048, K=4001, a="e5m2", b="e4m3", b_rows=1, out="fp32", temperature=False),
        # one served token with 20 alternatives
        dict(name="logprobs-one-token", op="logprobs", T=1, V=151936, m=1, top_n=20, src="fp32", mask="none", pad=0, temperature=False),
        # a scored rollout: the replayed token, the entropy and a few alternatives
        dict(name="logprobs-rollout", op="logprobs", T=4096, V=152064, m=1, top_n=8, src="bf16", mask="none", pad=0, temperature=True),
        # a teacher's 64 tokens a position, a third of the vocabulary masked, odd vocabulary and row stride
        dict(name="logprobs-teacher-ragged", op="logprobs", T=999, V=50021, m=64, top_n=64, src="fp16", mask="inf", pad=6, temperature=True),
        # the gradient of a policy loss with an entropy bonus
        dict(name="gradient-rollout", op="gradient", T=4096, V=152064, m=1, top_n=0, src="bf16", mask="none", pad=0, temperature=True, entropy=True),
        # the gradient of a distillation loss over a teacher's tokens and the student's own top ones
        dict(name="gradient-teacher-ragged", op="gradient", T=333, V=32771, m=64, top_n=16, src="fp32", mask="lowest", pad=1, temperature=True, entropy=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "logprobs", "gradient"])
    if op == "quantize":
        R, K = _log_uniform(rng, 1, 152064), _log_uniform(rng, 64, 16384)
        while R * K > 151936 * 4096:
            R = max(1, R // 2)
        return dict(op=op, R=R, K=K, src=rng.choice(["bf16", "bf16", "fp32", "fp16"]), to=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    block_rows=rng.choice([1, 1, 128]), transposed=rng.random() < 0.3)
    if op == "product":
        M, N, K = _log_uniform(rng, 1, 16384), _log_uniform(rng, 64, 152064), _log_uniform(rng, 64, 16384)
        while M * N * K > 4096 * 152064 * 5120 or M * N > 4096 * 152064:
            M = max(1, M // 2)
        a = rng.choice(["e4m3", "e4m3", "e5m2"])
        return dict(op=op, M=M, N=N, K=K, a=a, b="e4m3", b_rows=rng.choice([128, 128, 1]), out=rng.choice(["fp32", "fp32", "bf16"]),
                    temperature=rng.random() < 0.4)
    T, V = _log_uniform(rng, 1, 8192), _log_uniform(rng, 512, 262144)
    while T * V > 4096 * 152064:
        T = max(1, T // 2)
    c = dict(op=op, T=T, V=V, m=rng.choice([1, 1, 2, 8, 64]), top_n=rng.choice([0, 1, 5, 20, 64]), src=rng.choice(["fp32", "bf16", "bf16", "fp16"]),
             mask=rng.choice(["none", "none", "inf", "lowest"]), pad=rng.choice([0, 0, 1, 3, 8]), temperature=rng.random() < 0.7)
    if op == "gradient":
        c["entropy"] = rng.random() < 0.6
    return c


# ---------------------------------------------------------------- inputs


def _codes(gen, R, K, to, block_rows, spread):
    """An 8-bit matrix and its scales, as a user's program holds them: rows of a stride of whole 16 bytes."""
    dev = gen.device
    x = torch.randn(R, K, device=dev, generator=gen)
    if spread:  # gradients: most entries small, a few large
        x = x * torch.exp(torch.randn(R, 1, device=dev, generator=gen))
    q, scale = _quantize_plain(x, block_rows, to)
    ld = -(-K // 16) * 16
    held = torch.zeros(R, ld, dtype=torch.uint8, device=dev).view(FP8[to][0])
    held.view(torch.uint8)[:, :K] = q.view(torch.uint8)
    return held[:, :K], scale * (0.02 if spread else 1.0)


def _logits(gen, case):
    T, V, dt = case["T"], case["V"], FLOAT[case["src"]]
    dev = gen.device
    z = torch.randn(T, V + case["pad"], device=dev, generator=gen).mul_(2.0)
    hot = torch.randint(V, (T, 8), device=dev, generator=gen)  # the tokens that a context asks for
    z.scatter_add_(1, hot, 4.0 + 8.0 * torch.rand(T, 8, device=dev, generator=gen))
    if case["mask"] != "none":
        off = torch.rand(T, V + case["pad"], device=dev, generator=gen) < 1.0 / 3
        z.masked_fill_(off, -math.inf if case["mask"] == "inf" else torch.finfo(dt).min)
        if case["mask"] == "inf" and T > 2:
            z[T // 2] = -math.inf  # a row whose mask leaves nothing
    z = z.to(dt)[:, :V]
    tokens = torch.randint(V, (T, case["m"]), device=dev, generator=gen)
    first = torch.where(torch.rand(T, device=dev, generator=gen) < 0.8, z.argmax(1), hot[:, 1])
    tokens[:, 0] = first
    if case["m"] > 2:
        tokens[:, 1] = hot[:, 0]
        tokens[torch.rand(T, case["m"], device=dev, generator=gen) < 0.1] = -1  # shorter lists
        tokens[:, 2] = tokens[:, 0]  # the same token twice
    tau = torch.rand(T, device=dev, generator=gen) + 0.5 if case["temperature"] else None
    return z, tokens, tau


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "quantize":
        shape = (case["K"], case["R"]) if case["transposed"] else (case["R"], case["K"])
        x = torch.randn(shape, device=dev, generator=gen)
        x.mul_(torch.exp(torch.randn(shape[0], 1, device=dev, generator=gen)))
        x = x.to(FLOAT[case["src"]])
        s["x"] = x.t() if case["transposed"] else x
    elif case["op"] == "product":
        s["A"], s["a_scale"] = _codes(gen, case["M"], case["K"], case["a"], 1, case["a"] == "e5m2")
        s["B"], s["b_scale"] = _codes(gen, case["N"], case["K"], case["b"], case["b_rows"], False)
        s["b_scale"] = s["b_scale"] / math.sqrt(case["K"])
        s["tau"] = torch.rand(case["M"], device=dev, generator=gen) + 0.5 if case["temperature"] else None
    else:
        s["z"], s["tokens"], s["tau"] = _logits(gen, case)
        if case["op"] == "gradient":
            T = case["T"]
            f = _logprobs_plain(s["z"], s["tokens"], s["tau"], case["top_n"])
            s["saved"] = {k: f[k] for k in ("logit_max", "log_sum", "entropy", "flags", "top_id")}
            s["g"] = torch.randn(T, case["m"], device=dev, generator=gen)
            s["g_entropy"] = 0.1 * torch.randn(T, device=dev, generator=gen) if case["entropy"] else None
            s["g_top"] = torch.randn(T, case["top_n"], device=dev, generator=gen) if case["top_n"] else None
    return s


# ---------------------------------------------------------------- plain forms


def _blocks(x, block_rows, value=0.0):
    """[R, K] padded to whole blocks, as [row blocks, block_rows, K blocks, 128]."""
    R, K = x.shape
    Rb, Kb = -(-R // block_rows), -(-K // BLOCK)
    x = torch.nn.functional.pad(x, (0, Kb * BLOCK - K, 0, Rb * block_rows - R), value=value)
    return x.reshape(Rb, block_rows, Kb, BLOCK)


def _quantize_plain(x, block_rows, to):
    """scale = largest finite magnitude of the block / largest code (1 where that is 0); code = x / scale, rounded to
    nearest even, at most the largest code; what is not finite becomes NaN."""
    dt, top = FP8[to]
    R, K = x.shape
    b = _blocks(x.float(), block_rows)
    finite = torch.isfinite(b)
    scale = torch.where(finite, b.abs(), 0.0).amax((1, 3)) / top
    scale = torch.where(scale > 0, scale, 1.0)
    y = (b / scale[:, None, :, None]).clamp(-top, top)
    y = torch.where(finite, y, math.nan)
    return y.reshape(y.shape[0] * y.shape[1], -1)[:R, :K].to(dt), scale


def _spread(scale, R, K, block_rows):
    """One scale per element."""
    return scale.repeat_interleave(block_rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :K]


def _product_plain(s):
    A = s["A"].float() * _spread(s["a_scale"], s["M"], s["K"], 1)
    B = s["B"].float() * _spread(s["b_scale"], s["N"], s["K"], s["b_rows"])
    C = A @ B.t()
    if s["tau"] is not None:
        C = C / s["tau"][:, None]
    return C.to(FLOAT[s["out"]])


def _keys(z):
    """int64 keys whose descending order is (logit descending, id ascending): the bits of the fp32 logit, monotone, above
    the id counted from the end."""
    V = z.shape[1]
    bits = (z + 0.0).view(torch.int32)  # + 0.0: minus zero counts as zero
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
    return (bits << 32) + (V - 1 - torch.arange(V, device=z.device))


def _logprobs_plain(z, tokens, tau, top_n):
    T, V = z.shape
    z = z.float()
    tau = torch.ones(T, device=z.device) if tau is None else tau
    zmax = z.amax(1)
    empty = zmax == -math.inf
    d = (z - torch.where(empty, 0.0, zmax)[:, None]) / tau[:, None]  # s - max s: 0 or less
    e = torch.exp(d)
    total = e.sum(1)
    log_sum = torch.where(empty, -math.inf, torch.log(total))
    entropy = torch.log(total) - torch.where(e > 0, e * d, 0.0).sum(1) / total
    given = torch.gather(d, 1, tokens.clamp(min=0)) - log_sum[:, None]
    given = torch.where(empty[:, None], -math.inf, given)
    out = dict(logprob=torch.where(tokens < 0, 0.0, given), entropy=torch.where(empty, 0.0, entropy), logit_max=zmax, log_sum=log_sum,
               lse=torch.where(empty, -math.inf, zmax / tau + log_sum), flags=torch.where(empty, 8, 0).to(torch.int32))
    n = min(top_n, V)
    if n:
        key = torch.topk(_keys(z), n, dim=1).values
        ids = V - 1 - (key & 0xFFFFFFFF)
        lp = torch.gather(d, 1, ids) - log_sum[:, None]
        none = torch.gather(z, 1, ids) == -math.inf
        out["top_id"] = torch.nn.functional.pad(torch.where(none, -1, ids), (0, top_n - n), value=-1)
        out["top_logprob"] = torch.nn.functional.pad(torch.where(none, -math.inf, lp), (0, top_n - n), value=-math.inf)
    else:
        out["top_id"] = torch.empty(T, 0, dtype=torch.int64, device=z.device)
        out["top_logprob"] = torch.empty(T, 0, device=z.device)
    return out


def _gradient_plain(s):
    z, f = s["z"].float(), s["saved"]
    T, V = z.shape
    tau = torch.ones(T, device=z.device) if s["tau"] is None else s["tau"]
    live = (f["flags"] & 2 == 0) & (f["flags"] & 8 == 0)
    lp = (z - torch.where(live, f["logit_max"], 0.0)[:, None]) / tau[:, None] - torch.where(live, f["log_sum"], 0.0)[:, None]
    p = torch.exp(lp)
    ids, g = s["tokens"], s["g"]
    if s["g_top"] is not None:
        ids, g = torch.cat([ids, f["top_id"]], 1), torch.cat([g, s["g_top"]], 1)
    at = ids.clamp(min=0)
    g = torch.where((ids >= 0) & (torch.gather(z, 1, at) > -math.inf), g, 0.0)
    dz = -p * g.sum(1)[:, None]
    if s["g_entropy"] is not None:
        dz -= s["g_entropy"][:, None] * torch.where(p > 0, p * (lp + f["entropy"][:, None]), 0.0)
    dz.scatter_add_(1, at, g)
    dz = dz / tau[:, None]
    return torch.where(live[:, None], dz, 0.0).to(s["z"].dtype)


# ---------------------------------------------------------------- one pass


def _run_own(s):
    import sampling_transform_lm_b200 as sts

    if s["op"] == "quantize":
        q, scale = sts.sts_block_quantize(s["x"], block_rows=s["block_rows"], dtype=FP8[s["to"]][0])
        return dict(q=q, scale=scale)
    if s["op"] == "product":
        return dict(C=sts.sts_block_scaled_product(s["A"], s["a_scale"], s["B"], s["b_scale"], temperature=s["tau"], out_dtype=FLOAT[s["out"]]))
    if s["op"] == "logprobs":
        logprob, f = sts.sts_token_logprobs(s["z"], s["tokens"], temperature=s["tau"], top_n=s["top_n"], entropy=True)
        return dict(logprob=logprob, entropy=f["entropy"], lse=f["lse"], top_id=f["top_id"], top_logprob=f["top_logprob"])
    return dict(dz=sts.sts_token_logprobs_backward(s["z"], s["tokens"], s["saved"], s["g"], grad_entropy=s["g_entropy"], grad_top=s["g_top"],
                                                   temperature=s["tau"]))


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "quantize":
        q, scale = _quantize_plain(state["x"], state["block_rows"], state["to"])
        return dict(q=q, scale=scale)
    if state["op"] == "product":
        return dict(C=_product_plain(state))
    if state["op"] == "logprobs":
        f = _logprobs_plain(state["z"], state["tokens"], state["tau"], state["top_n"])
        return {k: f[k] for k in ("logprob", "entropy", "lse", "top_id", "top_logprob")}
    return dict(dz=_gradient_plain(state))


def work(case):
    size = dict(fp32=4, bf16=2, fp16=2)
    if case["op"] == "quantize":
        R, K = case["R"], case["K"]
        blocks = -(-R // case["block_rows"]) * -(-K // BLOCK)
        return dict(bytes=R * K * (size[case["src"]] + 1) + 4 * blocks, flops=3 * R * K)
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        Kb = -(-K // BLOCK)
        scales = 4 * Kb * (M + -(-N // case["b_rows"]))
        return dict(bytes=(M + N) * K + scales + M * N * size[case["out"]] + (4 * M if case["temperature"] else 0), flops=2 * M * N * K)
    T, V, m, n = case["T"], case["V"], case["m"], case["top_n"]
    read = T * V * size[case["src"]] + T * m * 8 + (4 * T if case["temperature"] else 0)
    if case["op"] == "logprobs":  # a difference, an exponential, two sums, a comparison and the product of the entropy
        return dict(bytes=read + T * (4 * m + 8 + 12 * n), flops=6 * T * V)
    return dict(bytes=read + T * V * size[case["src"]] + T * (4 * m + 12 * n + 16 + (4 if case["entropy"] else 0)), flops=7 * T * V)


# ---------------------------------------------------------------- the definitions in 64 bits


def _round_to_code(y, to):
    """y to the nearest value of the 8-bit type, ties to the even one."""
    mant, low, top = (3, -6, 448.0) if to == "e4m3" else (2, -14, 57344.0)
    e = torch.frexp(y)[1].to(torch.float64) - 1.0
    step = torch.exp2(e.clamp(min=low) - mant)
    return (torch.round(y / step) * step).clamp(-top, top)


def _exact_quantize(x, block_rows, to):
    R, K = x.shape
    top = FP8[to][1]
    b = _blocks(x.double(), block_rows)
    scale = b.abs().amax((1, 3)) / top
    scale[scale == 0] = 1.0
    q = _round_to_code(b / scale[:, None, :, None], to)
    return dict(q=q.reshape(q.shape[0] * q.shape[1], -1)[:R, :K], scale=scale)


def _exact_forward(z, tau):
    """Scaled logits, their log normaliser (-inf where the mask leaves nothing) and the row's entropy."""
    s = z.double()
    if tau is not None:
        s = s / tau.double()[:, None]
    lse = torch.logsumexp(s, 1)
    lp = s - torch.where(lse == -math.inf, 0.0, lse)[:, None]
    p = torch.exp(lp)
    H = -(p * torch.where(p > 0, lp, 0.0)).sum(1)
    return s, lse, lp, p, H


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(s["x"], case["block_rows"], case["to"])
    if case["op"] == "product":
        A = (s["A"].double().reshape(case["M"], -1) * _spread(s["a_scale"].double(), case["M"], case["K"], 1))
        B = (s["B"].double().reshape(case["N"], -1) * _spread(s["b_scale"].double(), case["N"], case["K"], case["b_rows"]))
        C = A @ B.t()
        return dict(C=C if s["tau"] is None else C / s["tau"].double()[:, None])
    z, tokens, tau = s["z"], s["tokens"], s["tau"]
    T, V = z.shape
    sc, lse, lp, p, H = _exact_forward(z, tau)
    if case["op"] == "logprobs":
        given = torch.where(tokens < 0, 0.0, torch.gather(lp, 1, tokens.clamp(min=0)))
        n = min(case["top_n"], V)
        key = z.float() + 0.0
        val, at = torch.sort(key, dim=1, descending=True, stable=True)
        at = torch.where(val[:, :n] == -math.inf, -1, at[:, :n])
        top = torch.where(at < 0, -math.inf, torch.gather(lp, 1, at.clamp(min=0)))
        more = case["top_n"] - n
        return dict(logprob=given, entropy=H, lse=lse, top_id=torch.nn.functional.pad(at, (0, more), value=-1),
                    top_logprob=torch.nn.functional.pad(top, (0, more), value=-math.inf))
    # sum_j g_j (onehot_j - p) - g_H p (ln p + H), over the temperature
    ids, g = tokens, s["g"].double()
    if s["g_top"] is not None:
        ids, g = torch.cat([ids, s["saved"]["top_id"]], 1), torch.cat([g, s["g_top"].double()], 1)
    g = torch.where((ids >= 0) & (torch.gather(sc, 1, ids.clamp(min=0)) > -math.inf), g, 0.0)
    dz = torch.zeros(T, V, dtype=torch.float64, device=z.device).scatter_add_(1, ids.clamp(min=0), g)
    dz -= g.sum(1, keepdim=True) * p
    if s["g_entropy"] is not None:
        dz -= s["g_entropy"].double()[:, None] * p * (torch.where(p > 0, lp, 0.0) + H[:, None])
    if tau is not None:
        dz = dz / tau.double()[:, None]
    return dict(dz=torch.where((lse > -math.inf)[:, None], dz, 0.0))
