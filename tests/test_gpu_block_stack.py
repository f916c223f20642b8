"""The block-scaled products, the gated norms and AdamW as a training step
runs them together: each call against its definition on the buffers that the
step left, whole steps against each other."""
import pytest
import torch

from fp8_relu_mlp_b200 import _abi as A
from fp8_relu_mlp_b200.block import BlockScaledStack
import train_ops_ref as R

pytestmark = pytest.mark.gpu
BF, U8, F32, F64, F8 = torch.bfloat16, torch.uint8, torch.float32, torch.float64, torch.float8_e4m3fn
HALF, ROW = 2.0 ** -8, 2.0 ** -16


def stack(L, M, d, h, rows, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rnd(t, scale, add=0.0):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda") * scale + add)

    s = BlockScaledStack(L, M, d, h, rows)
    for l in range(L):
        rnd(s.W1[l], d ** -0.5)
        rnd(s.W2[l], h ** -0.5)
        rnd(s.w_pre[l], 0.1, 1)
        rnd(s.w_post[l], 0.1, 1)
        rnd(s.gate[l], 0.2, 0.5)
        rnd(s.alpha[l], 0.05, 0.9)
    rnd(s.r[0], 1.0)
    rnd(s.dr, 1e-3)
    s.refresh_caches()
    return s


def near(got, want, mag, rel=HALF):
    return bool(((got.to(F64) - want).abs() <= rel * want.abs() + 4 * ROW * mag + 1e-30).all())


@pytest.mark.parametrize("L,M,d,h,rows", [(2, 70, 144, 272, 33), (3, 300, 256, 512, None), (1, 1, 128, 400, 1),
                                          (2, 5, 768, 1024, 2)])
def test_forward_layer_by_layer(L, M, d, h, rows):
    s = stack(L, M, d, h, rows)
    s.forward()
    torch.cuda.synchronize()
    assert A.fp8mlp_get_device_status() == 0
    rows = s.rows
    for l in range(L):
        r, x, out, post = s.r[l].to(F64), s.x[l].to(F64), s.out[l].to(F64), s.post[l].to(F64)
        # x_l is the norm of r_l before r_l was rounded: r_l is within half a step of that
        rp = 1 / torch.sqrt((r * r).mean(1) + s.eps)
        xe = r * rp[:, None] * s.w_pre[l].to(F64)
        assert bool(((x - xe).abs() <= 2.1 * HALF * xe.abs() + HALF * xe.abs().amax(1, keepdim=True)).all())
        # post from x within the codes' half steps: 2^-4 of each product's factors
        W1, W2 = s.W1[l].to(F64), s.W2[l].to(F64)
        pre, mag = x @ W1.t(), x.abs() @ W1.abs().t()
        assert bool(((post.sqrt() - pre.clamp(min=0)).abs() <= 0.14 * mag + 1e-12).all())
        # out and r_{l+1} from the buffers
        oe, mag = post @ W2, post.abs() @ W2.abs()
        assert bool(((out - oe).abs() <= 0.14 * mag + 1e-12).all())
        rn, rpost, _, _ = R.norms_fwd(r, out, s.w_post[l].to(F64), s.gate[l].to(F64), rows, s.alpha[l].to(F64), None, s.eps)
        assert near(s.r[l + 1], rn, r.abs() + (rn - s.alpha[l].to(F64) * r).abs())
        assert near(s.rstd_post[l], rpost, rpost, 0)


@pytest.mark.parametrize("L,M,d,h,rows", [(2, 70, 144, 272, 33), (3, 300, 256, 512, None), (2, 5, 768, 1024, 1)])
def test_backward_is_the_chain_of_its_calls(L, M, d, h, rows):
    s = stack(L, M, d, h, rows, seed=3)
    s.forward()
    dr_top = s.dr.clone()
    s.backward()
    got = {k: [t.clone() for t in getattr(s, k)] for k in ("dW1", "dW2", "dw_pre", "dw_post", "dgate", "dalpha")}
    dr0 = s.dr.clone()
    # the same from the definitions in float64 over BF16 buffers, layer by layer
    dr, dX = dr_top, None
    for l in range(L - 1, -1, -1):
        f = lambda t: None if t is None else t.to(F64)
        pre = l + 1 < L
        rn, rpost, _, rpre = R.norms_fwd(f(s.r[l]), f(s.out[l]), f(s.w_post[l]), f(s.gate[l]), s.rows, f(s.alpha[l]), None,
                                         s.eps)
        want, mag = R.norms_bwd(f(s.r[l]), f(s.out[l]), f(s.w_post[l]), f(s.gate[l]), s.rows, f(s.alpha[l]),
                                f(s.rstd_post[l]), f(s.r[l + 1]), f(s.w_pre[l + 1]) if pre else None,
                                f(s.rstd_pre[l + 1]) if pre else None, f(dX), f(dr))
        for k, t in (("dw_post", got["dw_post"][l]), ("dgate", got["dgate"][l]), ("dalpha", got["dalpha"][l]),
                     ("dw_pre", got["dw_pre"][l + 1] if pre else None)):
            if t is not None:
                # dr and dX of the layers above came in rounded to BF16, here in another order of sums
                assert bool(((t.to(F64) - want[k]).abs() <= (2 * HALF + ROW) * mag[k] + 1e-30).all()), (k, l)
        dOut = want["dy"].to(BF)
        post = s.post[l].to(F64)
        dPre = (2 * post.sqrt() * (dOut.to(F64) @ s.W2[l].to(F64).t())).to(BF)
        for k, w in (("dW1", dPre.to(F64).t() @ s.x[l].to(F64)), ("dW2", post.t() @ dOut.to(F64))):
            assert float((got[k][l].to(F64) - w).norm()) <= 1e-2 * float(w.norm()), (k, l)
        dX = (dPre.to(F64) @ s.W1[l].to(F64)).to(BF)
        dr = want["dr"].to(BF)
    want, mag = R.norms_bwd(s.r[0].to(F64), None, None, None, 1, None, None, s.r[0].to(F64), s.w_pre[0].to(F64),
                            s.rstd_pre[0].to(F64), dX.to(F64), dr.to(F64))
    assert float((dr0.to(F64) - want["dr"]).norm()) <= 1e-2 * float(want["dr"].norm())
    assert float((got["dw_pre"][0].to(F64) - want["dw_pre"]).norm()) <= 1e-2 * float(want["dw_pre"].norm())


@pytest.mark.parametrize("bits,masters", [(8, True), (32, True), (8, False)])
def test_steps_captured_and_eager_are_the_same(bits, masters):
    runs = []
    for graph in (False, True):
        s = stack(2, 130, 256, 384, 50, seed=7)
        opt = s.optimizer(state_bits=bits, masters=masters, weight_decay=0.1, lr=1e-2, max_norm=0.5, seed=5)
        r0, dr = s.r[0].clone(), s.dr.clone()
        before = [w.clone() for w in s.W1]

        def step():
            s.r[0].copy_(r0)
            s.dr.copy_(dr)
            s.train_step(opt)

        step()
        if graph:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            g.replay()
            g.replay()
        else:
            step()
            step()
        torch.cuda.synchronize()
        assert opt.read_state()["step"] == 3 and A.fp8mlp_get_device_status() == 0
        assert all(not torch.equal(a, b) for a, b in zip(before, s.W1))
        # the caches are those of the weights
        for l in range(2):
            q, sc = R.quant_weight(s.W1[l].float())
            assert torch.equal(s.W1q[l], q.view(U8)) and torch.equal(s.w1s[l], sc)
        runs.append([t.clone() for k in ("W1", "W2", "w_pre", "w_post", "gate", "alpha", "r", "W1q", "W2q_t")
                     for t in getattr(s, k)] + [v for e in opt.entries for v in e.values() if v is not None])
    assert all(torch.equal(a.view(U8), b.view(U8)) for a, b in zip(*runs))


@pytest.mark.parametrize("handle,graph", [(False, False), (True, False), (False, True)])
def test_a_stack_on_a_stream_of_its_own(handle, graph):
    # weights and inputs are written on the current stream, which is busy while the calls are made
    L, M, d, h, rows, steps = 2, 130, 256, 384, 50, 3
    names = ("W1", "W2", "w_pre", "w_post", "gate", "alpha")
    kw = dict(state_bits=8, weight_decay=0.1, lr=1e-2, max_norm=0.5, seed=5)
    one = stack(L, M, d, h, rows, seed=7)
    start = {k: [t.clone() for t in getattr(one, k)] for k in names}
    r0, dr = one.r[0].clone(), one.dr.clone()
    opt = one.optimizer(**kw)
    for _ in range(steps):
        one.r[0].copy_(r0)
        one.dr.copy_(dr)
        one.train_step(opt)
    a = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()

    def busy():
        nonlocal a
        for _ in range(10):
            a = a @ a * 1e-3

    side = torch.cuda.Stream()
    busy()
    two = BlockScaledStack(L, M, d, h, rows, stream=side.cuda_stream if handle else side)
    for k in names:
        for t, w in zip(getattr(two, k), start[k]):
            t.copy_(w)
    two.refresh_caches()
    with torch.cuda.stream(side):
        busy()  # the masters are taken behind this
    opt2 = two.optimizer(**kw)

    def step():
        two.r[0].copy_(r0)
        two.dr.copy_(dr)
        two.train_step(opt2)

    busy()
    step()
    torch.cuda.synchronize()  # the next copies overwrite what a step on another stream reads
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        for _ in range(steps - 1):
            g.replay()
    else:
        for _ in range(steps - 1):
            busy()
            step()
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert opt2.read_state()["step"] == steps and A.fp8mlp_get_device_status() == 0
    for k in names + ("r", "W1q", "W2q_t"):
        assert all(torch.equal(x.view(U8), y.view(U8)) for x, y in zip(getattr(one, k), getattr(two, k))), k
    for x, y in zip(opt.entries, opt2.entries):
        assert all(torch.equal(x[k].view(U8), y[k].view(U8)) for k in x if x[k] is not None)
