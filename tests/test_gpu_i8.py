"""The 8-bit codes, their product and the minGRU modes on 8-bit weights,
against the oracle.

Tolerances.  Codes and scales are defined to the bit: equal.  A product is an
exact integer, rounded to fp32, times the rounded product of two scales: at
most 2^-24 each, relative, three times (below 2^-22); one more rounding of 2^-8
relative (half an ulp of 8 significant bits) when y is bf16.  The step's gates
follow from k and p of that accuracy through exp2 and rcp (one ulp each): a
relative error of sigma of a few 2^-23 plus 2^-22 |k|, taken as 2^-18 (1 + |g|
+ |h|) max(1, (|k| + |p|) / 8) on h' = h + z (g - h)."""

import numpy as np
import pytest
import torch

from oracle import mingru, quant, scalar
from tests.gpu_util import dev, host64, say

pytestmark = pytest.mark.gpu

sr = pytest.importorskip("scan_linear_rnn_amd")

F32_TOL, BF16_TOL = 2.0 ** -22, 2.0 ** -8 + 2.0 ** -22


def _host(t):
    return t.detach().float().cpu().numpy() if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


def _activations(rng, M, K):
    x = rng.standard_normal((M, K)).astype(np.float32)
    if K:
        x[:, rng.integers(0, K, max(1, K // 64))] *= 8
    return x


def _same_codes(q, s, x):
    q_ref, s_ref = quant.quantize_rows(x)
    assert q.dtype == torch.int8 and tuple(q.shape) == q_ref.shape
    assert np.array_equal(_host(s), s_ref, equal_nan=True)
    assert np.array_equal(_host(q), q_ref)


# ------------------------------------------------------------------- codes


@pytest.mark.parametrize("M,K", [(1, 1), (3, 127), (2, 128), (5, 129), (70, 1000), (257, 512),
                                 (300, 2048), (9, 4100), (2, 20000), (1, 131072), (4, 0), (0, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows(M, K, dtype):
    say(f"i8 rows {M}x{K} {dtype}")
    x = dev(_activations(np.random.default_rng([3000, M, K]), M, K), dtype)
    q, s = sr.quantize_rows(x)
    _same_codes(q, s, _host(x))


@pytest.mark.parametrize("K,N", [(1, 1), (127, 3), (128, 65), (1000, 130), (2048, 96), (3000, 20),
                                 (5000, 17), (0, 8), (16, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_columns(K, N, dtype):
    say(f"i8 columns {K}x{N} {dtype}")
    W = dev(np.random.default_rng([3010, K, N]).standard_normal((K, N)).astype(np.float32), dtype)
    q, s = sr.quantize_columns(W)
    _same_codes(q, s, _host(W).T.copy())


@pytest.mark.parametrize("M,K", [(3, 7), (2, 8), (5, 9), (40, 1001), (2100, 777), (7, 2049), (3, 4103), (2, 32767), (2, 33001)])
@pytest.mark.parametrize("start", [0, 1])
def test_bf16_rows_at_odd_elements(M, K, start):
    """Odd lengths, odd distances and odd starts, at the end of their memory."""
    say(f"i8 odd rows {M}x{K}+{start}")
    rng = np.random.default_rng([3011, M, K])
    held = torch.zeros(start + M * K, device="cuda", dtype=torch.bfloat16)
    held[start:] = dev(rng.standard_normal((M, K)).astype(np.float32), torch.bfloat16).reshape(-1)
    x = held[start:].view(M, K)
    _same_codes(*sr.quantize_rows(x), _host(x))


@pytest.mark.parametrize("K,N", [(1, 8), (5, 9), (300, 7), (1000, 1001), (2049, 50), (4097, 70), (4096, 515), (9000, 33), (513, 4100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_columns_at_odd_elements(K, N, dtype):
    say(f"i8 odd columns {K}x{N} {dtype}")
    rng = np.random.default_rng([3021, K, N])
    held = torch.zeros(1 + K * N, device="cuda", dtype=dtype)
    held[1:] = dev(rng.standard_normal((K, N)).astype(np.float32), dtype).reshape(-1)
    W = held[1:].view(K, N)
    _same_codes(*sr.quantize_columns(W), _host(W).T)
    wide = dev(rng.standard_normal((K, N + 3)).astype(np.float32), dtype)[:, 2:2 + N]
    _same_codes(*sr.quantize_columns(wide), _host(wide).T)


@pytest.mark.parametrize("K", [130, 3000, 5000])
def test_columns_of_zeros_not_finite_and_at_the_ends_of_the_range(K):
    say(f"i8 special columns K={K}")
    rng = np.random.default_rng([3022, K])
    W = rng.standard_normal((K, 200)).astype(np.float32)
    W[:, 3] = 0
    W[:, 64:96] = 0
    W[:, 100] *= 1e-38
    W[:, 101] *= 1e36
    W[K - 1, 120] = np.nan
    W[0, 130] = -np.inf
    W[:, 140] *= 1e-44
    _same_codes(*sr.quantize_columns(dev(W)), W.T)


@pytest.mark.parametrize("K", [1, 3, 4, 7, 8, 9, 127, 128, 129, 255, 256, 257, 383, 511, 512, 513])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_short_rows_of_all_kinds_side_by_side(K, dtype):
    """Rows of zeros, of NaNs and infinities and at the ends of the range among
    ordinary ones."""
    say(f"i8 short rows K={K} {dtype}")
    rng = np.random.default_rng([3015, K])
    x = rng.standard_normal((1003, K)).astype(np.float32)
    x[5:9] = 0
    x[17, K - 1], x[40, 0], x[41, K // 2] = np.nan, np.inf, -np.inf
    x[60] *= 1e-37
    x[61] *= 1e35
    x[1002] *= 1e-30
    t = dev(x, dtype)
    _same_codes(*sr.quantize_rows(t), _host(t))
    wide = dev(np.hstack([x, x[:, :1], x[:, :1], x[:, :1]]), dtype)[:, 1:1 + K]  # rows K + 3 apart
    _same_codes(*sr.quantize_rows(wide), _host(wide))


def test_rows_special_values_and_ties():
    say("i8 rows special values")
    K = 300
    x = np.zeros((9, K), np.float32)
    x[1] = -0.0
    x[2, 7], x[2, 9] = np.nan, 3.0
    x[3, 299], x[3, 0] = np.inf, 3.0
    x[4, 0] = -np.inf
    x[5, :4] = [1e-45, -1e-45, 0.0, 3e-45]             # the scale underflows
    x[6, :3] = [3e-43, -2e-43, 1e-45]                  # a subnormal scale: quotients past 127 clamp
    x[7, :6] = [127.0, 0.5, 1.5, 2.5, -0.5, -126.5]    # ties to even at scale 1
    x[8, :2] = [3.0e38, -3.4e38]
    q, s = sr.quantize_rows(dev(x))
    _same_codes(q, s, x)
    qc, sc = sr.quantize_columns(dev(x.T.copy()))
    _same_codes(qc, sc, x)
    b, sb = sr.quantize_rows(dev(np.ones((4, K), np.float32)))
    y = _host(sr.matmul_i8(q, s, b, sb))
    assert np.isnan(y[2:5]).all() and np.isfinite(y[[0, 1, 5, 6, 7]]).all()


def test_strided_and_higher_rank_inputs():
    say("i8 strided inputs")
    rng = np.random.default_rng(3020)
    base = dev(rng.standard_normal((12, 3, 700)).astype(np.float32))
    half = base[:, 1, 3:603]                            # rows 2100 apart, 4-byte aligned
    _same_codes(*sr.quantize_rows(half), _host(half.contiguous()))
    q, s = sr.quantize_rows(base[:, :, 1:600])
    assert q.shape == (12, 3, 640) and s.shape == (12, 3)
    _same_codes(q.view(36, 640), s.view(36), _host(base[:, :, 1:600].reshape(36, 599)))
    Wt = dev(rng.standard_normal((50, 700)).astype(np.float32)).t()   # column-major weight
    _same_codes(*sr.quantize_columns(Wt), _host(Wt.t().contiguous()))
    Ws = base[:, 0, 5:77]
    _same_codes(*sr.quantize_columns(Ws), _host(Ws.t().contiguous()))


# ----------------------------------------------------------------- product


def _operands(rng, M, K, N):
    a = rng.integers(-127, 128, (M, K)).astype(np.int8)
    b = rng.integers(-127, 128, (N, K)).astype(np.int8)
    sa = rng.uniform(0.001, 0.1, M).astype(np.float32)
    sb = rng.uniform(0.001, 0.1, N).astype(np.float32)
    return a, sa, b, sb


def _close(y, ref, tol):
    err = np.abs(host64(y) - ref)
    assert np.all(err <= tol * np.abs(ref)), float(np.max(err / np.maximum(np.abs(ref), 1e-300)))


SHAPES = [(1, 128, 1), (1, 2048, 130), (2, 512, 64), (15, 256, 100), (16, 384, 48), (17, 128, 33),
          (31, 2048, 96), (33, 640, 257), (63, 1024, 65), (64, 128, 64), (65, 1024, 1030),
          (127, 512, 129), (129, 256, 127), (300, 2048, 200), (256, 1024, 1024), (511, 384, 2049),
          (1500, 256, 700), (5, 0, 7)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product(M, K, N, dtype):
    say(f"i8 product {M}x{K}x{N} {dtype}")
    a, sa, b, sb = _operands(np.random.default_rng([3100, M, K, N]), M, K, N)
    y = sr.matmul_i8(dev(a, torch.int8), dev(sa), dev(b, torch.int8), dev(sb), out_dtype=dtype)
    assert y.dtype == dtype
    _close(y, quant.product(a, sa, b, sb), F32_TOL if dtype == torch.float32 else BF16_TOL)


@pytest.mark.parametrize("M,K,N", [(5000, 1024, 3000), (4100, 512, 4500), (20000, 128, 1100),
                                   (40000, 256, 520)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_product_every_element(M, K, N, dtype):
    """Against float64 products on the GPU (sums of integers below 2^53: exact)."""
    say(f"i8 large product {M}x{K}x{N} {dtype}")
    a, sa, b, sb = (dev(t, torch.int8 if t.dtype == np.int8 else torch.float32)
                    for t in _operands(np.random.default_rng([3110, M, K, N]), M, K, N))
    y = sr.matmul_i8(a, sa, b, sb, out_dtype=dtype).double()
    ref = (a.double() @ b.double().t().contiguous()) * (sa.double()[:, None] * sb.double())
    tol = F32_TOL if dtype == torch.float32 else BF16_TOL
    assert bool(((y - ref).abs() <= tol * ref.abs()).all())


@pytest.mark.parametrize("M,K,N", [(5000, 1024, 3001), (1000, 640, 4097), (9000, 384, 4000), (16390, 128, 2055),
                                   (300, 128, 4100), (2047, 1024, 1537), (700, 2048, 2600)])
def test_odd_widths_and_line_counts_every_element(M, K, N):
    """Rows of results at odd elements, tiles that end inside, one, three and
    five lines of depth: each kernel against float64, and the bytes around the
    results untouched."""
    say(f"i8 odd product {M}x{K}x{N}")
    a, sa, b, sb = (dev(t, torch.int8 if t.dtype == np.int8 else torch.float32)
                    for t in _operands(np.random.default_rng([3115, M, K, N]), M, K, N))
    ref = (a.double() @ b.double().t().contiguous()) * (sa.double()[:, None] * sb.double())
    for dtype, tol in ((torch.float32, F32_TOL), (torch.bfloat16, BF16_TOL)):
        big = torch.full(((M + 2) * N + 1,), -7.0, device="cuda", dtype=dtype)
        y = big[N + 1:N + 1 + M * N].view(M, N)      # starts at an odd element
        sr.matmul_i8(a, sa, b, sb, out=y)
        assert bool(((y.double() - ref).abs() <= tol * ref.abs()).all())
        assert bool((big[:N + 1] == -7).all() and (big[N + 1 + M * N:] == -7).all())


@pytest.mark.parametrize("M,K,N", [(64, 2048, 4096), (256, 2048, 4096), (1500, 2048, 1000), (4096, 1024, 4096),
                                   (3000, 1152, 3000)])
def test_products_repeat_bit_for_bit(M, K, N):
    """Forty calls in a row on alternating operands: a stage read before it
    has landed, or loaded before it has been read, would differ now and then."""
    say(f"i8 repeat {M}x{K}x{N}")
    sets = [[dev(t, torch.int8 if t.dtype == np.int8 else torch.float32)
             for t in _operands(np.random.default_rng([3118, M, i]), M, K, N)] for i in range(2)]
    refs = [(a.double() @ b.double().t().contiguous() * (sa.double()[:, None] * sb.double())).float()
            for a, sa, b, sb in sets]
    first = [sr.matmul_i8(*s) for s in sets]
    for y, ref in zip(first, refs):
        assert bool(((y - ref).abs() <= 2 * F32_TOL * ref.abs()).all())
    for rep in range(40):
        assert torch.equal(sr.matmul_i8(*sets[rep % 2]), first[rep % 2]), rep


def test_product_extreme_codes_at_the_deepest_k():
    """All codes 127 at K = 131072: the sum 127^2 K is just below 2^31."""
    say("i8 deepest product")
    K = 131072
    a = np.full((3, K), 127, np.int8)
    a[1] = -127
    b = np.full((40, K), 127, np.int8)
    one = np.ones(40, np.float32)
    y = sr.matmul_i8(dev(a, torch.int8), dev(one[:3]), dev(b, torch.int8), dev(one))
    _close(y, quant.product(a, one[:3], b, one), F32_TOL)


def test_product_strides_and_out():
    say("i8 product strides")
    rng = np.random.default_rng(3120)
    a, sa, b, sb = _operands(rng, 70, 512, 90)
    A, B = dev(a, torch.int8), dev(b, torch.int8)
    ref = quant.product(a[:, :256], sa, b[:, :256], sb)
    out = torch.full((70, 90), float("nan"), device="cuda")
    y = sr.matmul_i8(A[:, :256], dev(sa), B[:, :256], dev(sb), out=out)   # rows 512 bytes apart
    assert y is out
    _close(y, ref, F32_TOL)
    ref3 = sr.matmul_i8(A, dev(sa), B, dev(sb))
    y3 = sr.matmul_i8(A.view(7, 10, 512), dev(sa).view(7, 10), B, dev(sb))
    assert y3.shape == (7, 10, 90) and torch.equal(y3.view(70, 90), ref3)
    odd = torch.empty(70 * 512 + 1, dtype=torch.int8, device="cuda")[1:].view(70, 512)  # misaligned
    odd.copy_(A)
    assert torch.equal(sr.matmul_i8(odd, dev(sa), B, dev(sb)), ref3)


@pytest.mark.parametrize("M,K,N", [(3, 256, 100), (40, 256, 100), (200, 256, 300), (2200, 256, 2100)])
def test_product_writes_only_its_rows(M, K, N):
    """Output inside a larger buffer: what lies around it stays as it is."""
    say(f"i8 product bounds {M}x{K}x{N}")
    import ctypes
    a, sa, b, sb = _operands(np.random.default_rng([3130, M]), M, K, N)
    A, B, SA, SB = dev(a, torch.int8), dev(b, torch.int8), dev(sa), dev(sb)
    ref = sr.matmul_i8(A, SA, B, SB)
    for pad in (1, 4):
        big = torch.full((M + 2, N + pad), -7.0, device="cuda")
        inner = big[1:, :N]
        st = sr.raw_library().matmul_i8(M, N, K, A.data_ptr(), K, SA.data_ptr(), B.data_ptr(), K,
                                        SB.data_ptr(), inner.data_ptr(), N + pad, sr.SR_F32,
                                        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        assert torch.equal(big[1:M + 1, :N], ref)
        assert bool((big[0] == -7).all() and (big[M + 1] == -7).all() and (big[:, N:] == -7).all())


@pytest.mark.parametrize("N", range(1017, 1024))
def test_every_width_of_the_last_columns(N):
    """One to seven columns past the last 16 bytes, in tiles of 128 x 128 and
    of 256 x 256, against the narrow product's rows."""
    say(f"i8 last columns N={N}")
    M, K = 40000, 1024
    a, sa, b, sb = (dev(t, torch.int8 if t.dtype == np.int8 else torch.float32)
                    for t in _operands(np.random.default_rng([3140, N]), M, K, N))
    for dtype in (torch.float32, torch.bfloat16):
        for rows in (M, 2100):
            big = torch.full((rows * N + 9,), -7.0, device="cuda", dtype=dtype)
            y = big[4:4 + rows * N].view(rows, N)
            sr.matmul_i8(a[:rows], sa[:rows], b, sb, out=y)
            for at in (0, 1000, rows - 60):
                assert torch.equal(y[at:at + 60], sr.matmul_i8(a[at:at + 60], sa[at:at + 60], b, sb, out_dtype=dtype))
            ref = (a[:rows].float() @ b.float().t().contiguous()) * sa[:rows, None] * sb
            assert bool(((y.float() - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -20 * K * 127 * 127 * sa[:rows, None] * sb).all())
            assert bool((big[:4] == -7).all() and (big[4 + rows * N:] == -7).all())


@pytest.mark.parametrize("M,N", [(40, 700), (300, 8195)])
def test_rows_of_results_more_than_2_20_elements_apart(M, N):
    say(f"i8 far rows {M}x{N}")
    import ctypes
    K, far = 256, (1 << 20) + 3
    a, sa, b, sb = _operands(np.random.default_rng([3145, M]), M, K, N)
    A, B, SA, SB = dev(a, torch.int8), dev(b, torch.int8), dev(sa), dev(sb)
    for dtype, code in ((torch.float32, sr.SR_F32), (torch.bfloat16, sr.SR_BF16)):
        ref = sr.matmul_i8(A, SA, B, SB, out_dtype=dtype)
        big = torch.full((M, far), -7.0, device="cuda", dtype=dtype)
        st = sr.raw_library().matmul_i8(M, N, K, A.data_ptr(), K, SA.data_ptr(), B.data_ptr(), K,
                                        SB.data_ptr(), big.data_ptr(), far, code,
                                        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        assert torch.equal(big[:, :N], ref) and bool((big[:, N:] == -7).all())


def test_outputs_past_2_31_elements():
    say("i8 product past 2^31 outputs")
    M, K, N = 70000, 128, 32768
    g = torch.Generator(device="cuda")
    g.manual_seed(3140)
    a = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    b = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sa, sb = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    y = sr.matmul_i8(a, sa, b, sb, out_dtype=torch.bfloat16)
    for rows in (slice(0, 300), slice(65400, 65700), slice(69700, 70000)):
        ref = (a[rows].double() @ b.double().t().contiguous()) * (sa[rows].double()[:, None] * sb.double())
        assert bool(((y[rows].double() - ref).abs() <= BF16_TOL * ref.abs()).all())
    q, s = sr.quantize_rows(y)                           # and reading them back
    _same_codes(q[-3:], s[-3:], _host(y[-3:]))
    assert not bool(q[:, 0].eq(-128).any())


# -------------------------------------------------------------- minGRU modes


def _layer(rng, D_in, D_h, D_out):
    W_in = (rng.standard_normal((D_in, 2 * D_h)) / max(D_in, 1) ** 0.5).astype(np.float32)
    W_out = (rng.standard_normal((D_h, D_out)) / max(D_h, 1) ** 0.5).astype(np.float32) if D_out else None
    return W_in, W_out


def _gates(x, W_in, D_h):
    """k and p in float64 from the codes of x's rows and of W_in's columns."""
    kp = quant.product(*quant.quantize_rows(x), *quant.quantize_rows(W_in.T.copy()))
    return kp[:, :D_h], kp[:, D_h:]


def _h_close(h, k, p, h_prev, decay=1.0):
    z, g = scalar.sigmoid(k), scalar.g(p)
    hp = np.asarray(h_prev, np.float64) * decay
    ref = hp + z * (g - hp)
    tol = 2.0 ** -18 * (1 + np.abs(g) + np.abs(hp)) * np.maximum(1, (np.abs(k) + np.abs(p)) / 8)
    assert np.all(np.abs(host64(h) - ref) <= tol), float(np.max(np.abs(host64(h) - ref) / tol))


STEPS = [(1, 16, 16, 16), (2, 512, 512, 512), (16, 100, 33, 7), (17, 192, 200, 130), (33, 300, 64, 65),
         (64, 128, 65, 1), (130, 257, 100, 64), (256, 1024, 512, 700), (600, 64, 190, 33),
         (1030, 384, 1100, 200), (4100, 200, 513, 130)]


@pytest.mark.parametrize("B,D_in,D_h,D_out", STEPS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step(B, D_in, D_h, D_out, dtype):
    say(f"i8 step B={B} {D_in}->{D_h}->{D_out} {dtype}")
    rng = np.random.default_rng([3200, B, D_in, D_h])
    W_in, W_out = _layer(rng, D_in, D_h, D_out)
    x = dev(_activations(rng, B, D_in), dtype)
    h0 = rng.standard_normal((B, D_h)).astype(np.float32)
    wi, wo = sr.quantize_columns(dev(W_in)), sr.quantize_columns(dev(W_out))
    y, h = sr.mingru_step_i8(x, *wi, *wo, h_prev=dev(h0))
    _h_close(h, *_gates(_host(x), W_in, D_h), h0)
    assert y.dtype == dtype and y.shape == (B, D_out)
    y_ref = quant.product(*quant.quantize_rows(_host(h)), *quant.quantize_rows(W_out.T.copy()))
    _close(y, y_ref, F32_TOL if dtype == torch.float32 else BF16_TOL)
    h1 = sr.mingru_step_i8(x, *wi, h_prev=dev(h0))[0]      # no W_out: the state is the output
    assert torch.equal(h1, h)
    state = dev(h0)
    sr.mingru_step_i8(x, *wi, h_prev=state, h_next=state)  # in place
    assert torch.equal(state, h)
    z = sr.mingru_step_i8(x, *wi)[0]                       # absent state: zeros
    assert torch.equal(z, sr.mingru_step_i8(x, *wi, h_prev=torch.zeros_like(h))[0])


@pytest.mark.parametrize("B,D_in,D_h,D_out", [(1, 1, 1, 1), (2, 129, 100, 33), (3, 1000, 1023, 64), (4, 1024, 1025, 130),
                                              (4, 1030, 2048, 1000), (1, 2048, 4095, 17), (2, 4096, 4097, 96),
                                              (3, 4100, 64, 4100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step_of_few_tokens_equals_quantising_first(B, D_in, D_h, D_out, dtype):
    """Bit for bit: the same rows in a batch of more, and the output's product
    on codes of the state made by quantize_rows."""
    say(f"i8 tokens B={B} {D_in}->{D_h}->{D_out} {dtype}")
    rng = np.random.default_rng([3205, B, D_in, D_h])
    W_in, W_out = _layer(rng, D_in, D_h, D_out)
    wi, wo = sr.quantize_columns(dev(W_in)), sr.quantize_columns(dev(W_out))
    rows = _activations(rng, 21, D_in)
    rows[0] *= 1e-33      # a scale that takes the slow division
    h0 = rng.standard_normal((21, D_h)).astype(np.float32)
    decay = dict(decay_rate=dev(rng.uniform(0, 0.5, D_h).astype(np.float32)))
    gap = dev(rng.exponential(2.0, 21).astype(np.float32))
    for kw, gaps in ((dict(), None), (decay, gap)):
        if gaps is not None:
            kw = dict(kw, delta_t=gaps)
        many = sr.mingru_step_i8(dev(rows, dtype), *wi, h_prev=dev(h0), **kw)[0]
        if gaps is not None:
            kw = dict(kw, delta_t=gaps[:B])
        y, h = sr.mingru_step_i8(dev(rows[:B], dtype), *wi, *wo, h_prev=dev(h0[:B]), **kw)
        assert torch.equal(h, many[:B])
        assert torch.equal(y, sr.matmul_i8(*sr.quantize_rows(h), *wo, out_dtype=dtype))
    # a start of the rows that no dword begins at (bf16), and sums past a tile's rows
    held = torch.zeros(B * D_in + 1, device="cuda", dtype=dtype)
    held[1:] = dev(rows[:B], dtype).reshape(-1)
    h = sr.mingru_step_i8(held[1:].view(B, D_in), *wi, h_prev=dev(h0[:B]))[0]
    assert torch.equal(h, sr.mingru_step_i8(dev(rows, dtype), *wi, h_prev=dev(h0))[0][:B])


def test_few_tokens_with_empty_and_not_finite_rows():
    say("i8 tokens special rows")
    rng = np.random.default_rng(3206)
    D = 200
    W_in, W_out = _layer(rng, D, D, D)
    wi, wo = sr.quantize_columns(dev(W_in)), sr.quantize_columns(dev(W_out))
    x = _activations(rng, 4, D)
    x[0], x[1, 7], x[2, 199] = 0, np.nan, -np.inf
    h0 = np.zeros((4, D), np.float32)
    h0[3, 5] = np.nan
    y, h = sr.mingru_step_i8(dev(x), *wi, *wo, h_prev=dev(h0))
    assert torch.isfinite(h[0]).all() and torch.isnan(h[1:3]).all()
    assert torch.isnan(h[3, 5]) and torch.isfinite(h[3, :5]).all()
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1:]).all()


def test_step_with_time_decay():
    say("i8 step with decay")
    rng = np.random.default_rng(3210)
    for B in (3, 40, 200):
        D = 100
        W_in, _ = _layer(rng, D, D, 0)
        x, h0 = _activations(rng, B, D), rng.standard_normal((B, D)).astype(np.float32)
        rate = rng.uniform(0, 0.5, D).astype(np.float32)
        gap = rng.exponential(2.0, B).astype(np.float32)
        sat = torch.zeros(1, dtype=torch.int32, device="cuda")
        wi = sr.quantize_columns(dev(W_in))
        kw = dict(h_prev=dev(h0), decay_rate=dev(rate), saturated=sat)
        h = sr.mingru_step_i8(dev(x), *wi, delta_t=dev(gap), **kw)[0]
        gamma = np.exp(-rate[None, :].astype(np.float64) * gap[:, None].astype(np.float64))
        _h_close(h, *_gates(x, W_in, D), h0, gamma)
        assert int(sat) == 0
        gap[1] = 1e7
        h = sr.mingru_step_i8(dev(x), *wi, delta_t=dev(gap), **kw)[0]
        assert int(sat) == 1
        h_log = sr.mingru_step_i8(dev(x), *wi, delta_t=dev(np.expm1(np.ones(B)).astype(np.float32)),
                                  log1p_delta=True, **kw)[0]
        _h_close(h_log, *_gates(x, W_in, D), h0, np.exp(-rate.astype(np.float64)))


@pytest.mark.parametrize("B,D_in,D_h", [(200, 100, 90), (700, 256, 520), (1030, 384, 1100), (4100, 130, 513)])
@pytest.mark.parametrize("decay", [False, True])
def test_rows_of_a_large_step_equal_those_of_small_ones(B, D_in, D_h, decay):
    """Bit for bit: a row's state does not depend on the rows beside it."""
    say(f"i8 large step B={B} {D_in}->{D_h} decay={decay}")
    rng = np.random.default_rng([3215, B, D_in, D_h])
    W_in, _ = _layer(rng, D_in, D_h, 0)
    wi = sr.quantize_columns(dev(W_in))
    x = dev(_activations(rng, B, D_in))
    h0 = dev(rng.standard_normal((B, D_h)).astype(np.float32))
    rate = dev(rng.uniform(0, 0.5, D_h).astype(np.float32))
    gap = dev(rng.exponential(2.0, B).astype(np.float32))

    def step(rows):
        kw = dict(decay_rate=rate, delta_t=gap[rows]) if decay else {}
        return sr.mingru_step_i8(x[rows], *wi, h_prev=h0[rows], **kw)[0]

    h = step(slice(None))
    for at in sorted({0, 100, B // 2, B - 37}):
        assert torch.equal(h[at:at + 37], step(slice(at, at + 37)))
    _h_close(h, *_gates(_host(x), W_in, D_h), _host(h0),
             np.exp(-_host(rate)[None, :].astype(np.float64) * _host(gap)[:, None]) if decay else 1.0)


@pytest.mark.parametrize("B,T,D_in,D_h,D_out", [(2, 64, 16, 16, 16), (1, 1, 20, 30, 10),
                                                (3, 301, 100, 130, 70), (2, 1024, 512, 512, 512),
                                                (4, 0, 16, 16, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_forward(B, T, D_in, D_h, D_out, dtype):
    """The states against the sequential definition on the products' own k
    and p (rounded to bf16 where they are staged so): 1e-4 of the two terms
    of h for fp32, as every scan; y against the product of the codes of the
    states that the call without W_out returns."""
    say(f"i8 forward {B}x{T} {D_in}->{D_h}->{D_out} {dtype}")
    rng = np.random.default_rng([3220, T, D_h])
    W_in, W_out = _layer(rng, D_in, D_h, D_out)
    x = dev(_activations(rng, B * T, D_in).reshape(B, T, D_in), dtype)
    h0 = dev(rng.standard_normal((B, D_h)).astype(np.float32))
    wi, wo = sr.quantize_columns(dev(W_in)), sr.quantize_columns(dev(W_out))
    h, last = sr.mingru_forward_i8(x, *wi, h0=h0, return_last=True)
    assert h.dtype == torch.float32
    kp = sr.matmul_i8(*sr.quantize_rows(x), *wi, out_dtype=dtype)
    kp_ref = quant.product(*quant.quantize_rows(_host(x).reshape(B * T, D_in)),
                           *quant.quantize_rows(W_in.T.copy()))
    _close(kp.view(B * T, 2 * D_h), kp_ref, F32_TOL if dtype == torch.float32 else BF16_TOL)
    k, p = host64(kp)[..., :D_h], host64(kp)[..., D_h:]
    if T:
        ref = mingru.scan(k, p, host64(h0))
        carry, inp = mingru.scan_terms(k, p, host64(h0))
        assert np.all(np.abs(host64(h) - ref) <= 1e-4 * (carry + inp))
        assert torch.equal(last, h[:, -1])
    else:
        assert torch.equal(last, h0)
    y, last2 = sr.mingru_forward_i8(x, *wi, *wo, h0=h0, return_last=True)
    assert y.dtype == dtype and y.shape == (B, T, D_out) and torch.equal(last2, last)
    y_ref = quant.product(*quant.quantize_rows(_host(h).reshape(B * T, D_h)),
                          *quant.quantize_rows(W_out.T.copy())).reshape(B, T, D_out)
    _close(y, y_ref, F32_TOL if dtype == torch.float32 else BF16_TOL)


def test_layer_object_modes_agree():
    """The quantised layer's parallel mode and its token loop carry the same
    states (fp32 activations: k and p are the same numbers in both)."""
    say("i8 layer modes")
    g = torch.Generator()
    g.manual_seed(3230)
    layer = sr.MinGRU(96, generator=g, decay_rate=0.05)
    q = layer.quantized()
    x = torch.randn(3, 40, 96, generator=g).cuda()
    gaps = torch.rand(3, 40, generator=g).cuda()
    for dt in (None, gaps):
        y, last = q(x, None, return_next_prev_hidden=True, delta_t=dt)
        h, ys = torch.zeros(3, 96, device="cuda"), []
        for t in range(40):
            y_t, h = q(x[:, t], h, return_next_prev_hidden=True, delta_t=None if dt is None else dt[:, t])
            ys.append(y_t)
        assert float((h - last).abs().max()) <= 1e-4 * float(last.abs().max())
        # One code of h apart moves y by its weight: a bound of 1e-2 of y's size.
        assert float((torch.stack(ys, 1) - y).abs().max()) <= 1e-2 * float(y.abs().max())
        exact = layer(x, delta_t=dt)   # 8 bits against fp32: a percent or so
        assert float((y - exact).norm() / exact.norm()) < 0.03
    layer.W_in.mul_(0.5)
    old = q.W_in.data_ptr()
    q.requantize(layer)
    assert q.W_in.data_ptr() == old
    assert torch.equal(q.W_in_scale, sr.quantize_columns(layer.W_in)[1])


def test_operands_past_4_gib():
    """Codes of 4.6 GiB and a step's weights of just under 4 GiB: rows at
    their ends against the same rows alone."""
    say("i8 operands past 4 GiB")
    K = 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(3240)
    big = torch.randint(-127, 128, (1_200_000, K), dtype=torch.int8, device="cuda", generator=g)
    scale = torch.rand(big.shape[0], device="cuda", generator=g) + 0.1
    few, few_scale = big[1_000_000:1_000_003].clone(), scale[:3].clone()
    ends = (0, 524_280, big.shape[0] - 40)
    y = sr.matmul_i8(few, few_scale, big, scale)          # the weights are large
    for at in ends:
        assert torch.equal(y[:, at:at + 40], sr.matmul_i8(few, few_scale, big[at:at + 40], scale[at:at + 40]))
    y = sr.matmul_i8(big, scale, few, few_scale)          # the rows are
    for at in ends:
        assert torch.equal(y[at:at + 40], sr.matmul_i8(big[at:at + 40], scale[at:at + 40], few, few_scale))
    D, D_in = 131_000, 4 * K
    W, ws = big.view(-1, D_in)[:2 * D], scale[:2 * D] * 1e-4
    for B in (2, 40, 300):
        x = torch.randn(B, D_in, device="cuda", generator=g)
        h0 = torch.randn(B, D, device="cuda", generator=g)
        h = sr.mingru_step_i8(x, W, ws, h_prev=h0)[0]
        for at in (0, 65_530, D - 40):
            part = slice(at, at + 40)
            Wp = torch.cat([W[part], W[D + at:D + at + 40]])
            wsp = torch.cat([ws[part], ws[D + at:D + at + 40]])
            assert torch.equal(h[:, part], sr.mingru_step_i8(x, Wp, wsp, h_prev=h0[:, part].contiguous())[0])
    del big, W
    x = torch.randn(1_100_000, K, device="cuda", generator=g, dtype=torch.bfloat16)  # 8.4 GiB
    q, s = sr.quantize_rows(x)
    at = x.shape[0] - 50
    q_end, s_end = sr.quantize_rows(x[at:].clone())
    assert torch.equal(q[at:], q_end) and torch.equal(s[at:], s_end)


def test_another_stream_and_repeatability():
    say("i8 streams")
    rng = np.random.default_rng(3240)
    W_in, W_out = _layer(rng, 256, 256, 256)
    wi, wo = sr.quantize_columns(dev(W_in)), sr.quantize_columns(dev(W_out))
    x, h0 = dev(_activations(rng, 64, 256)), dev(rng.standard_normal((64, 256)).astype(np.float32))
    ref = sr.mingru_step_i8(x, *wi, *wo, h_prev=h0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            got = sr.mingru_step_i8(x, *wi, *wo, h_prev=h0)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_graph_replays_match_eager():
    say("i8 graph")
    rng = np.random.default_rng(3250)
    W_in, W_out = _layer(rng, 256, 256, 256)
    wi, wo = sr.quantize_columns(dev(W_in)), sr.quantize_columns(dev(W_out))
    xs = [dev(_activations(rng, 48, 256), torch.bfloat16) for _ in range(8)]
    h0 = dev(rng.standard_normal((48, 256)).astype(np.float32))

    def loop():
        h, y = h0, None
        for x in xs:
            y, h = sr.mingru_step_i8(x, *wi, *wo, h_prev=h)
        return y, h

    y_ref, h_ref = loop()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loop()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = loop()
    for rep in range(3):
        junk = loop()                       # eager work between replays
        torch.cuda.synchronize()
        y.zero_(), h.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, h_ref) and torch.equal(y, y_ref) and torch.equal(junk[1], h_ref), rep
