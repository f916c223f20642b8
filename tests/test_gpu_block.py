"""FP8 products with a scale for each block of 128 against plain definitions:
quantisers bit for bit, products within the fp32 accumulation bound."""
import numpy as np
import pytest
import torch

from fp8_relu_mlp_b200 import _abi as A
from gpu_util import Guarded
import train_ops_ref as R

pytestmark = pytest.mark.gpu
BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * scale).to(BF)


def wide(seed, M, K):
    """Values over many binades, with zero groups and outlier columns."""
    t = torch.randn(M, K, generator=gen(seed), device="cuda")
    t = t * torch.exp2(torch.randint(-30, 30, (M, 1), generator=gen(seed + 1), device="cuda").float())
    t[:, ::37] *= 50
    t[M // 2] = 0
    return t.to(BF)


def codes(t):
    """float8 -> bytes, the sign of zero dropped."""
    b = t.view(U8) if t.dtype != U8 else t
    return torch.where(b == 0x80, torch.zeros_like(b), b)


def quantize(x):
    M, K = x.shape
    q, s = Guarded((M, K), U8), Guarded((R.cdiv(K, 128), M), F32)
    A.fp8mlp_quantize_block(M, K, x, q.t, s.t)
    torch.cuda.synchronize()
    assert q.intact() and s.intact()
    return q.t.view(torch.float8_e4m3fn), s.t


def weight(W, both=True):
    N, K = W.shape
    kb, nb = R.cdiv(K, 128), R.cdiv(N, 128)
    q, s, qt, st = Guarded((N, K), U8), Guarded((kb, nb), F32), Guarded((K, N), U8), Guarded((nb, kb), F32)
    A.fp8mlp_weight_block_cache_refresh(N, K, W, q.t, s.t, qt.t if both else None, st.t if both else None)
    torch.cuda.synchronize()
    assert all(x.intact() for x in (q, s, qt, st))
    return q.t.view(torch.float8_e4m3fn), s.t, qt.t.view(torch.float8_e4m3fn), st.t


@pytest.mark.parametrize("M,K", [(1, 16), (2, 112), (15, 128), (17, 144), (33, 2064), (129, 512), (1000, 768)])
def test_quantiser_is_bit_exact(M, K):
    x = wide(M * 131 + K, M, K)
    q, s = quantize(x)
    wq, wsc = R.quant_rows(x.float())
    assert torch.equal(codes(q), codes(wq)) and torch.equal(s, wsc)


def test_quantiser_extremes():
    # all zero; BF16 subnormals (the scale stops at 2^120); the largest BF16;
    # an infinity and a NaN make their own group's scale NaN and no other's
    x = torch.zeros(8, 256, dtype=BF, device="cuda")
    x[1, :128] = 1e-39
    x[2, 5] = 3.3e38
    x[3, 200] = float("inf")
    x[4, 0], x[4, 1] = float("nan"), 3.0
    x[5, 127] = -float("inf")
    x[6, 130] = -1.0
    q, s = quantize(x)
    wq, wsc = R.quant_rows(x.float())
    assert torch.equal(torch.isnan(s), torch.isnan(wsc)) and torch.isnan(s).sum() == 3
    assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(wsc, nan=-1.0))
    ok = ~torch.isnan(s).t().repeat_interleave(128, dim=1)
    assert torch.equal(codes(q)[ok], codes(wq)[ok])
    assert s[0, 0] == 1 and s[0, 1] == 2.0 ** -120


@pytest.mark.parametrize("N,K", [(16, 16), (128, 128), (144, 272), (400, 112), (112, 2064), (768, 768)])
def test_weight_cache_is_bit_exact(N, K):
    W = wide(N * 7 + K, N, K)
    q, s, qt, st = weight(W)
    wq, wsc = R.quant_weight(W.float())
    assert torch.equal(codes(q), codes(wq)) and torch.equal(s, wsc)
    assert torch.equal(codes(qt), codes(q).t()) and torch.equal(st, s.t())
    q2, s2, _, _ = weight(W, both=False)
    assert torch.equal(codes(q2), codes(q)) and torch.equal(s2, s)


def within(got, exact, mag, terms):
    """bf16 rounding plus `terms` fp32 roundings of partial sums."""
    got = got.to(R.F64)
    bound = 2.0 ** -8 * exact.abs() + (1 + 2.0 ** -8) * terms * 2.0 ** -24 * mag + 1e-37
    return bool(((got - exact).abs() <= bound).all())


# (M, K, N): one token up to several tiles of both tile sizes, ragged in each direction
SHAPES = [(1, 16, 16), (1, 768, 2304), (2, 128, 128), (5, 144, 272), (8, 400, 48), (3, 1040, 2320), (4, 2064, 16), (6, 112, 144), (7, 4112, 48),
          (1, 768, 50304), (2, 16400, 32), (8, 4112, 48), (8, 2064, 4112), (16, 2064, 400), (17, 768, 144),
          (64, 256, 768), (127, 112, 128), (129, 1040, 400), (256, 128, 256), (257, 384, 1296), (300, 768, 3088),
          (2049, 272, 768), (4096, 256, 2048), (4999, 400, 2320)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_against_the_definition(M, K, N):
    x, W = wide(M + K, M, K), randn(N, N, K, scale=K ** -0.5)
    x = torch.where(x.abs() > 1e4, x.sign() * 1e4, x)
    Wq, ws, _, _ = weight(W, both=False)
    y, xq, xs = Guarded((M, N), BF), Guarded((M, K), U8), Guarded((R.cdiv(K, 128), M), F32)
    A.fp8mlp_linear_block(M, K, N, x, Wq, ws, xq.t, xs.t, y.t)
    torch.cuda.synchronize()
    assert y.intact() and xq.intact() and xs.intact() and A.fp8mlp_get_device_status() == 0
    q, s = quantize(x)
    assert torch.equal(codes(xq.t), codes(q)) and torch.equal(xs.t, s)
    exact, mag = R.product(q, s, Wq, ws)
    terms = K + 2 * R.cdiv(K, 128) + 4
    assert within(y.t, exact, mag, terms)
    # the same product from given codes
    y2 = Guarded((M, N), BF)
    A.fp8mlp_linear_fwd_block(M, K, N, q, s, Wq, ws, y2.t)
    torch.cuda.synchronize()
    assert y2.intact() and within(y2.t, exact, mag, terms)


@pytest.mark.parametrize("M,K,N", [(3, 144, 272), (300, 400, 256), (4999, 256, 1808)])
def test_input_gradient_through_the_transposed_cache(M, K, N):
    W, dY = randn(1, N, K, scale=0.05), randn(2, M, N, scale=1e-4)
    Wq, ws, Wqt, wst = weight(W)
    dX, q, s = torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(M, N, dtype=U8, device="cuda"), torch.empty(
        R.cdiv(N, 128), M, device="cuda")
    A.fp8mlp_linear_block(M, N, K, dY, Wqt, wst, q, s, dX)
    torch.cuda.synchronize()
    val = R.row_values(q.view(torch.float8_e4m3fn), s)
    Wv = R.weight_values(Wq, ws)
    assert within(dX, val @ Wv, val.abs() @ Wv.abs(), N + 2 * R.cdiv(N, 128) + 4)
    # against differences of the forward map: the layer is linear, so
    # <dX, v> = <dY, f(v)> up to the quantisation of dY (2^-4 an element)
    v = torch.randn(M, K, generator=gen(3), device="cuda", dtype=R.F64)
    fwd = v @ Wv.t()
    lhs, rhs = (dX.to(R.F64) * v).sum(), (dY.to(R.F64) * fwd).sum()
    slack = (dY.to(R.F64).abs() * 2.0 ** -4 * fwd.abs()).square().sum().sqrt() * 6 + 2.0 ** -8 * (
        dX.to(R.F64) * v).square().sum().sqrt() * 6
    assert abs(float(lhs - rhs)) <= float(slack)


@pytest.mark.parametrize("M,d,h", [(1, 16, 16), (1, 768, 1024), (7, 144, 272), (2, 1040, 112), (3, 128, 144),
                                   (4, 2320, 400), (5, 272, 656), (6, 16, 1040), (8, 512, 2064), (8, 4112, 48), (16, 256, 144), (130, 128, 400),
                                   (513, 272, 1040), (3000, 256, 2064)])
def test_up_projection_and_mlp(M, d, h):
    x, W1, W2 = randn(M, M, d), randn(2, h, d, scale=d ** -0.5), randn(3, h, d, scale=h ** -0.5)
    W1q, w1s, _, _ = weight(W1)
    _, _, W2qt, w2st = weight(W2)
    xq, xs = quantize(x)
    kh = R.cdiv(h, 128)
    post, pq, ps = Guarded((M, h), BF), Guarded((M, h), U8), Guarded((kh, M), F32)
    A.fp8mlp_up_proj_block(M, d, h, xq, xs, W1q, w1s, post.t, pq.t, ps.t)
    torch.cuda.synchronize()
    assert post.intact() and pq.intact() and ps.intact() and A.fp8mlp_get_device_status() == 0
    acc, mag = R.product(xq, xs, W1q, w1s)
    e = (d + 2 * R.cdiv(d, 128) + 4) * 2.0 ** -24 * mag  # of acc
    lo = (acc - e).clamp(min=0).square() * (1 - 2.0 ** -22)
    hi = (acc + e).clamp(min=0).square() * (1 + 2.0 ** -22)
    p = post.t.to(R.F64)
    assert bool(((p >= lo * (1 - 2.0 ** -8)) & (p <= hi * (1 + 2.0 ** -8))).all())
    # the scale maps the block's maximum, known to [lo, hi], onto 448
    def top(t):
        z = torch.zeros(M, kh * 128, dtype=R.F64, device="cuda")
        z[:, :h] = t
        return z.view(M, kh, 128).amax(2).t()
    tl, th = top(lo), top(hi)
    live = th > 0
    s = ps.t.to(R.F64)
    assert bool((s[live] >= tl[live] / 448 * (1 - 2.0 ** -22)).all())
    assert bool((s[live & (tl > 0)] <= th[live & (tl > 0)] / 448 * (1 + 2.0 ** -22)).all())
    # the codes stand for post within half a step (2^-4 of the value, 2^-10 of the scale near zero)
    val = R.row_values(pq.t.view(torch.float8_e4m3fn), ps.t)
    srow = s.t().repeat_interleave(128, dim=1)[:, :h]
    slack = 2.0 ** -20 * hi + 2.0 ** -10 * srow
    assert bool(((val >= lo * (1 - 2.0 ** -4) - slack) & (val <= hi * (1 + 2.0 ** -4) + slack)).all())
    # down-projection from exactly these codes, and the whole forward
    out, xq2, xs2 = Guarded((M, d), BF), torch.empty(M, d, dtype=U8, device="cuda"), torch.empty_like(xs)
    p2, pq2, ps2 = (torch.empty_like(t.t) for t in (post, pq, ps))
    A.fp8mlp_mlp_fwd_block(M, d, h, x, W1q, w1s, W2qt, w2st, xq2, xs2, p2, pq2, ps2, out.t)
    torch.cuda.synchronize()
    assert out.intact() and torch.equal(codes(xq2), codes(xq)) and torch.equal(xs2, xs)
    assert torch.equal(p2, post.t) and torch.equal(pq2, pq.t) and torch.equal(ps2, ps.t)
    exact, mag = R.product(pq.t.view(torch.float8_e4m3fn), ps.t, W2qt, w2st)
    assert within(out.t, exact, mag, h + 2 * kh + 4)


@pytest.mark.parametrize("M", [2, 300])
def test_nan_and_infinity_reach_the_rows_they_belong_to(M):
    d, h = 256, 384
    x = randn(5, M, d)
    x[1, 130] = float("inf")
    W = randn(6, h, d, scale=0.05)
    Wq, ws, _, _ = weight(W)
    xq, xs = quantize(x)
    y = torch.empty(M, h, dtype=BF, device="cuda")
    A.fp8mlp_linear_fwd_block(M, d, h, xq, xs, Wq, ws, y)
    post, pq, ps = torch.empty_like(y), torch.empty(M, h, dtype=U8, device="cuda"), torch.empty(3, M, device="cuda")
    A.fp8mlp_up_proj_block(M, d, h, xq, xs, Wq, ws, post, pq, ps)
    torch.cuda.synchronize()
    for t in (y, post, ps.t()):
        bad = torch.isnan(t)
        assert bad[1].all() and bad.sum() == bad[1].numel()


def test_empty_batch_writes_nothing():
    y = Guarded((4, 16), BF)
    q = torch.empty(16, 16, dtype=U8, device="cuda")
    s = torch.empty(4, device="cuda")
    before = y.t.clone()
    A.fp8mlp_linear_block(0, 16, 16, y.t, q, s, q, s, y.t)
    A.fp8mlp_mlp_fwd_block(0, 16, 16, y.t, q, s, q, s, q, s, y.t, q, s, y.t)
    torch.cuda.synchronize()
    assert torch.equal(y.t.view(torch.int16), before.view(torch.int16)) and y.intact()


@pytest.mark.parametrize("M", [4, 700])
def test_captured_replayed_and_on_another_stream(M):
    d, h = 256, 512
    x, W1, W2 = randn(1, M, d), randn(2, h, d, scale=0.06), randn(3, h, d, scale=0.04)
    W1q, w1s, _, _ = weight(W1)
    _, _, W2qt, w2st = weight(W2)

    def buffers():
        return (torch.empty(M, d, dtype=U8, device="cuda"), torch.empty(2, M, device="cuda"),
                torch.empty(M, h, dtype=BF, device="cuda"), torch.empty(M, h, dtype=U8, device="cuda"),
                torch.empty(4, M, device="cuda"), torch.empty(M, d, dtype=BF, device="cuda"))

    a, b = buffers(), buffers()
    A.fp8mlp_mlp_fwd_block(M, d, h, x, W1q, w1s, W2qt, w2st, *a)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    xin = x.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(g1):
        A.fp8mlp_mlp_fwd_block(M, d, h, xin, W1q, w1s, W2qt, w2st, *b)
    c = buffers()
    with torch.cuda.graph(g2):
        A.fp8mlp_mlp_fwd_block(M, d, h, xin, W1q, w1s, W2qt, w2st, *c)
    other = randn(9, M, d)
    xin.copy_(other)
    g1.replay()
    xin.copy_(x)
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    for u, v, w in zip(a, b, c):
        assert torch.equal(u.view(U8), v.view(U8)) and torch.equal(u.view(U8), w.view(U8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    e = buffers()
    A.fp8mlp_mlp_fwd_block(M, d, h, x, W1q, w1s, W2qt, w2st, *e, stream=side)
    side.synchronize()
    assert torch.equal(e[-1], a[-1])


def test_offsets_beyond_32_bits():
    # 2^31 + elements in x, its codes and y; the last rows are checked
    M, K, N = 2 ** 31 // 768 + 1000, 768, 16
    x = torch.empty(M, K, dtype=BF, device="cuda").fill_(0.5)
    tail = randn(4, 300, K)
    x[-300:] = tail
    q = torch.empty(M, K, dtype=U8, device="cuda")
    s = torch.empty(6, M, device="cuda")
    Wq, ws, _, _ = weight(randn(5, N, K, scale=0.05))
    y = torch.empty(M, N, dtype=BF, device="cuda")
    A.fp8mlp_linear_block(M, K, N, x, Wq, ws, q, s, y)
    torch.cuda.synchronize()
    wq, wsc = R.quant_rows(tail.float())
    assert torch.equal(codes(q[-300:]), codes(wq)) and torch.equal(s[:, -300:], wsc)
    exact, mag = R.product(wq, wsc, Wq, ws)
    assert within(y[-300:], exact, mag, K + 16)
    del x, q, y
    # and in the output
    M, K, N = 2 ** 31 // 2048 + 300, 16, 2048
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[-100:] = tail[:100, :K]
    Wq, ws, _, _ = weight(randn(6, N, K))
    q, s = torch.empty(M, K, dtype=U8, device="cuda"), torch.empty(1, M, device="cuda")
    y = torch.empty(M, N, dtype=BF, device="cuda")
    A.fp8mlp_linear_block(M, K, N, x, Wq, ws, q, s, y)
    torch.cuda.synchronize()
    exact, mag = R.product(q[-100:].view(torch.float8_e4m3fn), s[:, -100:], Wq, ws)
    assert within(y[-100:], exact, mag, K + 8) and not y[:1000].any()


@pytest.mark.parametrize("M,K,N", [(300, 256, 256), (8000, 384, 1808)])
def test_a_stalled_load_ends_with_a_status(M, K, N):
    x, W = randn(1, M, K), randn(2, N, K)
    Wq, ws, _, _ = weight(W)
    q, s = quantize(x)
    y = torch.empty(M, N, dtype=BF, device="cuda")
    A.fp8mlp_set_wait_timeout_ns(20_000_000)
    A.fp8mlp_set_debug_flags(A.DEBUG_STALL_PRODUCER)
    try:
        A.fp8mlp_linear_fwd_block(M, K, N, q, s, Wq, ws, y)
        assert A.fp8mlp_get_device_status() & A.STATUS_TIMEOUT
    finally:
        A.fp8mlp_set_debug_flags(0)
        A.fp8mlp_set_wait_timeout_ns(2_000_000_000)
        A.fp8mlp_clear_device_status()
    A.fp8mlp_linear_fwd_block(M, K, N, q, s, Wq, ws, y)
    torch.cuda.synchronize()
    exact, mag = R.product(q, s, Wq, ws)
    assert within(y, exact, mag, K + 8) and A.fp8mlp_get_device_status() == 0


def test_short_and_misplaced_buffers_are_refused():
    M, K, N = 4, 128, 256
    x, W = randn(1, M, K), randn(2, N, K)
    Wq, ws, _, _ = weight(W)
    q, s = quantize(x)
    y = torch.empty(M, N, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="y: "):
        A.fp8mlp_linear_fwd_block(M, K, N, q, s, Wq, ws, y[:3])
    with pytest.raises(ValueError, match="xs: "):
        A.fp8mlp_linear_fwd_block(M, K, N, q, s[:, :3].contiguous(), Wq, ws, y)
    with pytest.raises(ValueError, match="contiguous"):
        A.fp8mlp_linear_fwd_block(M, K, N, q, s, Wq, ws, torch.empty(N, M, dtype=BF, device="cuda").t())
    with pytest.raises(ValueError, match="CUDA"):
        A.fp8mlp_linear_fwd_block(M, K, N, q, s, Wq, ws, y.cpu())
    with pytest.raises(A.Fp8MlpError, match="aligned"):
        A.fp8mlp_linear_fwd_block(M, K, N, q, s, Wq, ws, torch.empty(M * N + 1, dtype=BF, device="cuda")[1:])


@pytest.mark.parametrize("M", [3, 200])
def test_the_mlp_may_write_over_its_input(M):
    d, h = 144, 272
    x, W1, W2 = randn(3, M, d), randn(4, h, d), randn(5, h, d)
    W1q, w1s, _, _ = weight(W1)
    _, _, W2q_t, w2s_t = weight(W2)

    def run(out):
        t = lambda r, c, dt: torch.empty(r, c, dtype=dt, device="cuda")  # noqa: E731
        A.fp8mlp_mlp_fwd_block(M, d, h, src, W1q, w1s, W2q_t, w2s_t, t(M, d, U8), t(2, M, F32), t(M, h, BF), t(M, h, U8),
                               t(3, M, F32), out)
        torch.cuda.synchronize()
        return out
    src = x
    want = run(torch.empty_like(x))
    src = x.clone()
    assert torch.equal(run(src), want)
    with pytest.raises(A.Fp8MlpError, match="y overlaps x"):
        sq = torch.zeros(M, d, dtype=BF, device="cuda")
        A.fp8mlp_linear_block(M, d, d, sq, W1q[:d].contiguous(), w1s, torch.empty(M, d, dtype=U8, device="cuda"),
                              torch.empty(2, M, device="cuda"), sq)


@pytest.mark.parametrize("M,K,N,one", [(1, 768, 2304, True), (1, 4096, 50304, True), (1, 16, 16, True), (4, 2048, 1024, True),
                                       (8, 512, 16384, False), (8, 128, 50304, False), (6, 768, 8192, False),
                                       (2, 16, 50304, False), (9, 64, 64, False)])
def test_few_rows_take_the_faster_form(M, K, N, one):
    # one launch where the pass over the weights is faster, two where the tensor cores are
    x = randn(M, M, K)
    Wq = torch.randint(0, 0x70, (N, K), dtype=U8, device="cuda", generator=gen(1))
    ws = torch.rand(R.cdiv(K, 128), R.cdiv(N, 128), device="cuda", generator=gen(2)) * 1e-2
    xq, xs, y = torch.empty(M, K, dtype=U8, device="cuda"), torch.empty(R.cdiv(K, 128), M, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
    n0 = A.fp8mlp_kernel_launch_count()
    A.fp8mlp_linear_block(M, K, N, x, Wq, ws, xq, xs, y)
    assert A.fp8mlp_kernel_launch_count() - n0 == (1 if one else 2)
    # from codes the same form, bit for bit
    again = torch.empty_like(y)
    A.fp8mlp_linear_fwd_block(M, K, N, xq, xs, Wq, ws, again)
    torch.cuda.synchronize()
    assert torch.equal(y, again) and A.fp8mlp_get_device_status() == 0
    exact, mag = R.product(xq.view(torch.float8_e4m3fn), xs, Wq.view(torch.float8_e4m3fn), ws)
    assert within(y, exact, mag, K + 2 * R.cdiv(K, 128) + 4)


def test_the_whole_mlp_repeats_itself():
    M, d, h = 2000, 1024, 4096
    x, W1, W2 = randn(M, M, d), randn(2, h, d, scale=d ** -0.5), randn(3, h, d, scale=h ** -0.5)
    W1q, w1s, _, _ = weight(W1)
    _, _, W2qt, w2st = weight(W2)
    first = None
    for i in range(8):
        o = [torch.full(s, 0x55, dtype=U8, device="cuda") for s in ((M, d), (M, 32), (M, 2 * h), (M, h), (M, 128), (M, 2 * d))]
        A.fp8mlp_mlp_fwd_block(M, d, h, x, W1q, w1s, W2qt, w2st, o[0], o[1], o[2], o[3], o[4], o[5])
        first = first or o
        assert all(torch.equal(a, b) for a, b in zip(first, o))
