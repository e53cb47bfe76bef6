"""What the 8-bit head's and the token log probabilities' entry points refuse, on the host: nothing here reaches a
device. The pointers are made up, so the file runs only where there is no GPU to follow one by mistake."""

import ctypes

import pytest
import torch

import sampling_transform_lm_b200 as sts
from sampling_transform_lm_b200 import _BlockOperand, _TokenRows, _TokenStats

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: host checks only")

OK, NULL, SHAPE, DTYPE, WORKSPACE = 0, 1, 2, 3, 9
F32, BF16, F16, E4M3, E5M2 = range(5)
P = 0x10000  # an address that is aligned for everything


@pytest.fixture(scope="module")
def lib():
    return sts.load()


def _quantize(lib, R=4, K=256, x=P, xt=BF16, sr=256, sk=1, br=1, qt=E4M3, q=P, q_ld=256, scale=P, s_ld=2):
    return lib.sts_block_quantize(R, K, x, xt, sr, sk, br, qt, q, q_ld, scale, s_ld, None)


@pytest.mark.parametrize("change,status", [
    (dict(R=-1), SHAPE), (dict(K=0), SHAPE), (dict(R=1 << 31), SHAPE), (dict(br=2), SHAPE), (dict(br=64), SHAPE),
    (dict(xt=E4M3), DTYPE), (dict(xt=9), DTYPE), (dict(qt=BF16), DTYPE), (dict(sr=255), SHAPE), (dict(sr=300, sk=2), SHAPE),
    (dict(sr=1, sk=3), SHAPE), (dict(q_ld=255), SHAPE), (dict(s_ld=1), SHAPE), (dict(x=None), NULL), (dict(q=None), NULL),
    (dict(scale=None), NULL), (dict(R=0, x=None, q=None, scale=None), OK), (dict(sr=-256), SHAPE)])
def test_quantize_refusals(lib, change, status):
    assert _quantize(lib, **change) == status


@pytest.mark.parametrize("change", [dict(x=P + 1), dict(x=P + 2, xt=F32), dict(x=P + 1, xt=F16), dict(scale=(1 << 42) + 1), dict(scale=(1 << 42) + 2),
                                    dict(x=P + 1, sr=1, sk=4), dict(x=P + 3, br=128)])
def test_quantize_refuses_what_is_not_aligned(lib, change):
    assert _quantize(lib, **dict(dict(q=1 << 41, scale=1 << 42), **change)) == SHAPE


def _bytes(at, n, pitch, width):
    return {b for i in range(n) for b in range(at + i * pitch, at + i * pitch + width)}


def _share(R, K, x, es, ld, transposed, q, q_ld, scale, s_ld, br):
    a = _bytes(x, K if transposed else R, ld * es, (R if transposed else K) * es)
    b = _bytes(q, R, q_ld, K)
    c = _bytes(scale, -(-R // br), s_ld * 4, -(-K // 128) * 4)
    return bool(a & b or a & c or b & c)


@pytest.mark.parametrize("change,status", [
    (dict(q=P, scale=1 << 40), SHAPE),  # in place
    (dict(q=P + 4 * 512 - 1, scale=1 << 40), SHAPE),  # x's last byte
    (dict(q=1 << 40, scale=P), SHAPE), (dict(q=1 << 40, scale=(1 << 40) + 252), SHAPE),
    (dict(sr=512, q=P + 512, q_ld=1024, scale=P + 768, s_ld=256), None),  # a record a row: source, codes, scales
    (dict(sr=512, q=P + 511, q_ld=1024, scale=P + 768, s_ld=256), SHAPE),
    (dict(sr=512, q=P + 512, q_ld=1024, scale=P + 764, s_ld=256), SHAPE),
    (dict(sr=512, q=P - 256, q_ld=1024, scale=P + 512, s_ld=256), None),
    (dict(sr=512, q=P - 255, q_ld=1024, scale=1 << 40), SHAPE),
    (dict(sr=512, q=P + 512, q_ld=512, scale=1 << 40), SHAPE),  # other pitches: the second row's codes meet x's second row
    (dict(sr=512, q=P + 512, q_ld=2048, scale=1 << 40), None)])
def test_quantize_refuses_results_inside_the_source_or_each_other(lib, change, status):
    args = dict(dict(q_ld=256, s_ld=2, sr=256), **change)
    shares = _share(4, 256, P, 2, args["sr"], False, args["q"], args["q_ld"], args["scale"], args["s_ld"], 1)
    assert shares == (status == SHAPE)
    got = _quantize(lib, **change)
    assert (got == SHAPE) == shares and (shares or got not in (OK, NULL, DTYPE))


def test_quantize_tells_overlap_byte_by_byte(lib):
    """Any small layout is refused exactly when a byte is shared."""
    import random

    rng = random.Random(0)
    told = [0, 0]
    for _ in range(3000):
        R, K = rng.randint(1, 5), rng.randint(1, 20)
        br, tr = rng.choice([1, 128]), rng.random() < 0.4
        ld = rng.randint(R if tr else K, 40)
        q_ld, s_ld = rng.randint(K, 90), rng.randint(1, 22)
        x, q, scale = P, P + rng.randint(-80, 300), P + 4 * rng.randint(-30, 120)
        if tr and ld == 1:
            continue
        got = _quantize(lib, R=R, K=K, x=x, sr=1 if tr else ld, sk=ld if tr else 1, br=br, q=q, q_ld=q_ld, scale=scale, s_ld=s_ld)
        shares = _share(R, K, x, 2, ld, tr, q, q_ld, scale, s_ld, br)
        assert (got == SHAPE) == shares, (R, K, br, tr, ld, q_ld, s_ld, q - P, scale - P)
        told[shares] += 1
    assert min(told) > 300


def _operand(rows=40, q=P, dtype=E4M3, ld=256, scale=P, sr=2, sk=1, block_rows=1):
    return _BlockOperand(q, dtype, rows, ld, scale, sr, sk, block_rows)


def _product(lib, a={}, b={}, K=256, C=P, ct=F32, ldc=40, acc=0, ws=None, ws_bytes=0):
    A, B = _operand(**a), _operand(**b)
    return lib.sts_block_scaled_product(ctypes.byref(A), ctypes.byref(B), K, None, C, ct, ldc, acc, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(K=0), SHAPE), (dict(a=dict(dtype=BF16)), DTYPE), (dict(b=dict(dtype=F32)), DTYPE), (dict(ct=F16), DTYPE),
    (dict(ct=BF16, acc=1), DTYPE), (dict(a=dict(block_rows=128)), SHAPE), (dict(b=dict(block_rows=64)), SHAPE),
    (dict(a=dict(ld=240)), SHAPE), (dict(a=dict(ld=264)), SHAPE), (dict(b=dict(q=P + 8)), SHAPE), (dict(b=dict(ld=257)), SHAPE),
    (dict(a=dict(scale=P + 2)), SHAPE), (dict(a=dict(sr=-1)), SHAPE), (dict(b=dict(rows=-1)), SHAPE), (dict(ldc=39), SHAPE),
    (dict(C=None), NULL), (dict(C=P + 2), SHAPE), (dict(a=dict(q=None)), NULL), (dict(b=dict(scale=None)), NULL),
    (dict(ws=P, ws_bytes=255), WORKSPACE), (dict(ws=P + 16, ws_bytes=4096), WORKSPACE), (dict(K=1 << 31), SHAPE),
    (dict(a=dict(rows=0, q=None, scale=None), C=None), OK), (dict(b=dict(rows=0, q=None, scale=None), C=None), OK)])
def test_product_refusals(lib, change, status):
    assert _product(lib, **change) == status


def test_product_refuses_missing_operands(lib):
    a = _operand()
    assert lib.sts_block_scaled_product(None, ctypes.byref(a), 256, None, P, F32, 40, 0, None, 0, None) == NULL
    assert lib.sts_block_scaled_product(ctypes.byref(a), None, 256, None, P, F32, 40, 0, None, 0, None) == NULL


def _rows(logits=P, dtype=F32, T=4, V=100, ld=100, tokens=P, m=2, tokens_ld=2, temperature=None, top_n=3):
    return _TokenRows(logits, dtype, T, V, ld, tokens, m, tokens_ld, temperature, top_n)


STATS = dict(logit_max=P, log_sum=P, lse=P, entropy=P, flags=P, top_id=P, top_logprob=P)

BAD_ROWS = [
    (dict(dtype=E4M3), DTYPE), (dict(T=-1), SHAPE), (dict(V=0), SHAPE), (dict(ld=99), SHAPE), (dict(m=513), SHAPE),
    (dict(m=-1), SHAPE), (dict(top_n=65), SHAPE), (dict(top_n=-1), SHAPE), (dict(tokens_ld=1), SHAPE), (dict(logits=None), NULL),
    (dict(tokens=None), NULL), (dict(logits=P + 2), SHAPE), (dict(V=1 << 31), SHAPE), (dict(T=1 << 30), SHAPE),
    (dict(T=0, logits=None, tokens=None), OK)]


@pytest.mark.parametrize("change,status", BAD_ROWS)
def test_token_logprobs_refusals(lib, change, status):
    r, s = _rows(**change), _TokenStats(**STATS)
    assert lib.sts_token_logprobs(ctypes.byref(r), P, ctypes.byref(s), None) == status


@pytest.mark.parametrize("missing,top_n", [("top_id", 3), ("top_logprob", 3)])
def test_token_logprobs_needs_its_outputs(lib, missing, top_n):
    r, s = _rows(top_n=top_n), _TokenStats(**dict(STATS, **{missing: None}))
    assert lib.sts_token_logprobs(ctypes.byref(r), P, ctypes.byref(s), None) == NULL
    s = _TokenStats(**STATS)
    assert lib.sts_token_logprobs(ctypes.byref(r), None, ctypes.byref(s), None) == NULL
    assert lib.sts_token_logprobs(ctypes.byref(r), P, None, None) == NULL
    assert lib.sts_token_logprobs(None, P, ctypes.byref(s), None) == NULL


def _backward(lib, rows={}, stats={}, g=P, h=P, gt=P, out=1 << 40, ot=F32, ld=100):
    r, s = _rows(**rows), _TokenStats(**dict(STATS, **stats))
    return lib.sts_token_logprobs_backward(ctypes.byref(r), ctypes.byref(s), g, h, gt, out, ot, ld, None)


@pytest.mark.parametrize("change,status", [(dict(rows=c), s) for c, s in BAD_ROWS] + [
    (dict(ot=E4M3), DTYPE), (dict(ld=99), SHAPE), (dict(out=None), NULL), (dict(out=(1 << 40) + 2), SHAPE),
    (dict(stats=dict(logit_max=None)), NULL), (dict(stats=dict(log_sum=None)), NULL), (dict(stats=dict(flags=None)), NULL),
    (dict(stats=dict(entropy=None)), NULL), (dict(stats=dict(top_id=None)), NULL),
    (dict(out=P + 4), SHAPE), (dict(out=P, ot=BF16), SHAPE), (dict(out=P, ld=101), SHAPE), (dict(out=P + 4 * 399), SHAPE)])
def test_backward_refusals(lib, change, status):
    assert _backward(lib, **change) == status


@pytest.mark.parametrize("name,off", [("logit_max", 2), ("log_sum", 1), ("lse", 3), ("entropy", 2), ("flags", 2), ("top_id", 4),
                                      ("top_logprob", 1)])
def test_misaligned_statistics_are_refused(lib, name, off):
    far = dict(out=1 << 40)
    r, s = _rows(), _TokenStats(**dict(STATS, **{name: P + off}))
    assert lib.sts_token_logprobs(ctypes.byref(r), P, ctypes.byref(s), None) == SHAPE
    assert _backward(lib, stats={name: P + off}, **far) == SHAPE


@pytest.mark.parametrize("change", [dict(rows=dict(tokens=P + 4)), dict(rows=dict(temperature=P + 2)), dict(g=P + 2), dict(h=P + 1),
                                    dict(gt=P + 3)])
def test_misaligned_rows_and_gradients_are_refused(lib, change):
    assert _backward(lib, **change) == SHAPE
    if "rows" in change:
        r, s = _rows(**change["rows"]), _TokenStats(**STATS)
        assert lib.sts_token_logprobs(ctypes.byref(r), P, ctypes.byref(s), None) == SHAPE
    r, s = _rows(), _TokenStats(**STATS)
    assert lib.sts_token_logprobs(ctypes.byref(r), P + 2, ctypes.byref(s), None) == SHAPE


def test_a_misaligned_temperature_of_the_product_is_refused(lib):
    A, B = _operand(), _operand()
    assert lib.sts_block_scaled_product(ctypes.byref(A), ctypes.byref(B), 256, P + 2, P, F32, 40, 0, None, 0, None) == SHAPE


def test_binding_refusals():
    bf = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(sts.StsError) as e:
        sts.sts_block_quantize(bf)
    assert "CUDA" in str(e.value)
    for bad in (dict(dtype=torch.int8), dict(block_rows=32)):
        with pytest.raises(sts.StsError):
            sts.sts_block_quantize(bf, **bad)
    with pytest.raises(sts.StsError) as e:
        sts.sts_block_quantize(torch.zeros(4, 256, dtype=torch.float64))
    assert e.value.status == DTYPE
    with pytest.raises(sts.StsError):
        sts.sts_block_quantize(bf[:, ::2][::2])
    for view in (torch.ones(1, 1).expand(5, 1), torch.ones(1, 4).expand(5, 4), torch.ones(4, 1).expand(4, 5)):
        with pytest.raises(sts.StsError) as e:  # a broadcast view has nothing behind its rows
            sts.sts_block_quantize(view)
        assert e.value.status == SHAPE and ("stride" in str(e.value) or "CUDA" in str(e.value))
    q = bf.to(torch.float8_e4m3fn)
    s = torch.ones(4, 2)
    for a, sa, b, sb, status in ((bf, s, q, s, DTYPE), (q, s[:3], q, s, SHAPE), (q, s, q, s[:, :1], SHAPE), (q, s.double(), q, s, DTYPE),
                                 (q, torch.ones(1, 2), q, s, SHAPE), (q, s, q[:, :128], s[:, :1], SHAPE)):
        with pytest.raises(sts.StsError) as e:
            sts.sts_block_scaled_product(a, sa, b, sb)
        assert e.value.status == status
    with pytest.raises(sts.StsError) as e:
        sts.sts_block_scaled_product(q, s, q, s, accumulate=True)
    assert e.value.status == NULL
    z = torch.zeros(4, 100)
    for tokens in (torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), torch.zeros(4, 2, 2, dtype=torch.int64)):
        with pytest.raises(sts.StsError):
            sts.sts_token_logprobs(z, tokens)
    with pytest.raises(sts.StsError) as e:
        sts.sts_token_logprobs(z.double(), None)
    assert e.value.status == DTYPE
    with pytest.raises(sts.StsError):
        sts.sts_token_logprobs(z, None, temperature=torch.ones(3))
    with pytest.raises(sts.StsError):
        sts.sts_token_logprobs(z, None, top_n=-1)


@pytest.mark.parametrize("lost,given", [("entropy", "grad_entropy"), ("top_id", "grad_top"), ("flags", None), ("log_sum", None)])
def test_the_gradient_says_what_the_saved_scalars_lack(lost, given):
    T, V, n = 3, 50, 2
    saved = dict(logit_max=torch.zeros(T), log_sum=torch.zeros(T), flags=torch.zeros(T, dtype=torch.int32), entropy=torch.zeros(T),
                 top_id=torch.zeros(T, n, dtype=torch.int64))
    grads = dict(grad_entropy=torch.zeros(T), grad_top=torch.zeros(T, n))
    for broken in ({k: v for k, v in saved.items() if k != lost}, dict(saved, **{lost: None})):
        with pytest.raises(sts.StsError) as e:
            sts.sts_token_logprobs_backward(torch.zeros(T, V), torch.zeros(T, dtype=torch.int64), broken, torch.zeros(T),
                                            **({given: grads[given]} if given else {}))
        assert e.value.status == NULL and lost in str(e.value)


@pytest.mark.parametrize("top_n", [-1, 65, 10 ** 9, 10 ** 12])
def test_too_many_alternatives_are_refused_before_they_are_allocated(top_n):
    with pytest.raises(sts.StsError) as e:
        sts.sts_token_logprobs(torch.zeros(4, 100), None, top_n=top_n)
    assert e.value.status == SHAPE and "top_n" in str(e.value)


def test_the_bf16_entry_points_still_refuse_an_8_bit_head():
    H = torch.zeros(4, 64, dtype=torch.bfloat16)
    W = torch.zeros(100, 64, dtype=torch.float8_e4m3fn)
    one = torch.ones(4)
    with pytest.raises(sts.StsError) as e:
        sts.sts_forward(H, W, torch.zeros(4, dtype=torch.int64), one, one.int(), one, one)
    assert e.value.status == DTYPE
