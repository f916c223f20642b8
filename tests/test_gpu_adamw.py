"""AdamW over many tensors against the step in fp32, operation by operation
(bit for bit), and against float64; the gradient norm against float64."""
import pytest
import torch

from fp8_relu_mlp_b200 import _abi as A
from fp8_relu_mlp_b200.optim import AdamW
import train_ops_ref as R

pytestmark = pytest.mark.gpu
BF, U8, F32, F8 = torch.bfloat16, torch.uint8, torch.float32, torch.float8_e4m3fn
HYPER = dict(b1=0.9, b2=0.95, eps=1e-8)


def tensors(sizes, bits, master, seed=0):
    """CPU values of each tensor: weights, gradient, moments as after some steps."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in sizes:
        mag = torch.exp(1.5 * torch.randn(n, generator=g)) * 1e-3
        t = dict(p=torch.randn(n, generator=g) * 0.02, g=torch.randn(n, generator=g) * mag,
                 m=0.3 * torch.randn(n, generator=g) * mag, v=mag * mag)
        if not master:
            t["p"] = t["p"].to(BF).float()
        if bits == 8:
            t["mq"], t["ms"] = R.quant_state(t["m"], torch.full((n,), 0.5), False)
            t["vq"], t["vs"] = R.quant_state(t["v"].sqrt(), torch.full((n,), 0.5), True)
        out.append(t)
    return out


def padded(x, dtype):
    """On the GPU with 256 guard bytes behind, 16-byte aligned."""
    raw = torch.full((x.numel() * torch.empty(0, dtype=dtype).element_size() + 256,), 0xA5, dtype=U8, device="cuda")
    t = raw[:-256].view(dtype)
    t.copy_(x.to(dtype))
    return t, raw


def build(ts, bits, master, copy=True, lr=1e-3, seed=7, step=4, max_norm=None, wd=0.1, lr_mult=None):
    opt = AdamW(state_bits=bits, lr=lr, betas=(HYPER["b1"], HYPER["b2"]), eps=HYPER["eps"], seed=seed, step_count=step,
                max_norm=max_norm)
    raws = []

    def put(x, dtype):
        t, raw = padded(x, dtype)
        raws.append(raw)
        return t

    for i, t in enumerate(ts):
        st = {"m": put(t["m"] if bits == 32 else t["mq"], F32 if bits == 32 else F8),
              "v": put(t["v"] if bits == 32 else t["vq"], F32 if bits == 32 else F8)}
        if bits == 8:
            st.update(m_scale=put(t["ms"], F32), v_scale=put(t["vs"], F32))
        opt.add(put(t["g"], F32), master=put(t["p"], F32) if master else None,
                weight=put(t["p"], BF) if copy or not master else None, weight_decay=wd,
                lr_mult=1.0 if lr_mult is None else lr_mult[i], state=st)
    return opt, raws


def expect(t, i, bits, master, step, lr, seed, coef=1.0, wd=0.1, lr_mult=1.0):
    """The step by torch on the GPU, whose fp32 division and square root are
    the correctly rounded ones (those of its vectorised CPU code are not
    always)."""
    t = {k: v.cuda() for k, v in t.items()}
    m = t["m"] if bits == 32 else R.state_values(t["mq"], t["ms"])
    u = None if bits == 32 else R.state_values(t["vq"], t["vs"])
    v = t["v"] if bits == 32 else u * u
    p, m, v = R.adamw(t["p"], t["g"], m, v, step, lr, wd, coef=coef, lr_mult=lr_mult, **HYPER)
    bits32 = R.random_bits(p.numel(), i, step, seed, device="cuda")
    out = dict(p=p, w=p.to(BF) if master else R.bf16_stochastic(p, R.mix32(bits32 ^ 0x5BD1E995) & 0xFFFF).to(BF))
    if bits == 32:
        out.update(m=m, v=v)
    else:
        out["m"], out["ms"] = R.quant_state(m, (bits32 & 0xFFFF).float() * 2.0 ** -16, False)
        out["v"], out["vs"] = R.quant_state(v.sqrt(), (bits32 >> 16).float() * 2.0 ** -16, True)
    return {k: v.cpu() for k, v in out.items()}


def same(e, want, bits, master):
    assert torch.equal(e["m"].float().cpu(), want["m"]) and torch.equal(e["v"].float().cpu(), want["v"])
    if bits == 8:
        assert torch.equal(e["m_scale"].cpu(), want["ms"]) and torch.equal(e["v_scale"].cpu(), want["vs"])
    if master:
        assert torch.equal(e["master"].cpu(), want["p"])
    if e["weight"] is not None:
        assert torch.equal(e["weight"].cpu(), want["w"])


SIZES = [1, 2, 3, 4, 5, 127, 128, 129, 1000, 4095, 4096, 4097, 0, 30001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master,copy", [(True, True), (True, False), (False, True)])
def test_step_is_the_fp32_step(bits, master, copy):
    ts = tensors(SIZES, bits, master)
    mult = [1.0 + 0.25 * (i % 3) for i in range(len(ts))]
    opt, raws = build(ts, bits, master, copy, lr_mult=mult)
    opt.step()
    torch.cuda.synchronize()
    assert opt.read_state() == dict(lr=R.f32(1e-3), step=5, seed=7, skipped=0)
    for i, (t, e) in enumerate(zip(ts, opt.entries)):
        same(e, expect(t, i, bits, master, 5, 1e-3, 7, lr_mult=mult[i]), bits, master)
    assert all(bool((r[-256:] == 0xA5).all()) for r in raws)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_takes(bits):
    sizes = [(37 * i) % 900 for i in range(300)]  # empty ones among them
    ts = tensors(sizes, bits, True)
    opt, raws = build(ts, bits, True)
    n0 = A.fp8mlp_kernel_launch_count()
    opt.step()
    assert A.fp8mlp_kernel_launch_count() - n0 == 2
    torch.cuda.synchronize()
    assert opt.read_state()["step"] == 5
    for i, (t, e) in enumerate(zip(ts, opt.entries)):
        same(e, expect(t, i, bits, True, 5, 1e-3, 7), bits, True)
    assert all(bool((r[-256:] == 0xA5).all()) for r in raws)


def test_many_steps_from_zero_against_float64():
    n = 3000
    g = torch.Generator().manual_seed(3)
    p = torch.randn(n, generator=g) * 0.02
    grads = [torch.randn(n, generator=g) * 1e-3 for _ in range(30)]
    opt = AdamW(state_bits=32, lr=1e-3, betas=(0.9, 0.95))
    gt, mt = torch.empty(n, device="cuda"), p.cuda()
    opt.add(gt, master=mt, weight_decay=0.1)
    P, m, v = p.double(), torch.zeros(n).double(), torch.zeros(n).double()
    for t, gr in enumerate(grads, 1):
        gt.copy_(gr)
        opt.step()
        P, m, v = R.adamw64(P, gr, m, v, t, 1e-3, 0.1, 0.9, 0.95, 1e-8)
    torch.cuda.synchronize()
    # 30 steps of size <= 2 lr each, every one within some 16 roundings of itself and of p; betas rounded to fp32
    tol = 30 * (16 * 2.0 ** -24 * (P.abs().max() + 2e-3) + 2e-3 * 2.0 ** -21)
    assert float((mt.cpu().double() - P).abs().max()) <= float(tol)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [True, False])
def test_eight_bit_states_follow_the_fp32_run(bits, master):
    # a constant gradient: m -> g, sqrt(v) -> |g|, and the weight moves by about lr a step,
    # however small one step's change of the state is next to a code's step
    n, steps, lr = 4096, 120, 1e-3
    g = torch.Generator().manual_seed(1)
    grad = torch.randn(n, generator=g).sign() * (0.5 + torch.rand(n, generator=g)) * 1e-3
    opt = AdamW(state_bits=bits, lr=lr, betas=(0.9, 0.999), seed=11)
    w = torch.zeros(n, device="cuda")
    w16 = torch.zeros(n, dtype=BF, device="cuda")
    e = opt.add(grad.cuda(), master=w if master else None, weight=w16)
    for _ in range(steps):
        opt.step()
    torch.cuda.synchronize()
    got = (w if master else w16.float()).cpu()
    ratio = (got / (-lr * steps * grad.sign())).double()
    # every step is lr (1 +- the codes' rounding, 2^-3 of m and of sqrt(v) at most), and independent over elements
    assert abs(float(ratio.mean()) - 1) < 0.03
    sv = (e["v"].float().cpu() if bits == 8 else e["v"].cpu().sqrt())
    if bits == 8:
        sv = R.state_values(sv, e["v_scale"].cpu())
    want = (grad.double().square() * (1 - 0.999 ** steps)).sqrt()
    assert abs(float((sv.double() / want).mean()) - 1) < 0.05


def test_moments_decay_without_gradient():
    # nearest rounding would hold sqrt(v) where it is (0.975 of it is nearer to it than to the next code)
    n = 12800
    opt = AdamW(state_bits=8, lr=0.0, betas=(0.9, 0.95), seed=5)
    grad = torch.ones(n, device="cuda")
    e = opt.add(grad, master=torch.zeros(n, device="cuda"))
    opt.step()
    grad.zero_()
    grad[::128] = 1.0  # holds each block's scale
    for _ in range(40):
        opt.step()
    torch.cuda.synchronize()
    u = R.state_values(e["v"].float().cpu(), e["v_scale"].cpu())
    rest = u[torch.arange(n) % 128 != 0]
    # E sqrt(v) = sqrt(0.05) 0.95^(40/2), the codes' noise averaged over 12700 elements
    want = 0.05 ** 0.5 * 0.95 ** 20
    assert 0.85 * want < float(rest.mean()) < 1.25 * want and bool((rest > 0).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step(bits):
    ts = tensors([5, 1000, 40000, 16385], bits, True)
    opt, _ = build(ts, bits, True, max_norm=0.01)
    opt.step()
    torch.cuda.synchronize()
    norm = sum(float(t["g"].double().square().sum()) for t in ts) ** 0.5
    got = opt.norm.cpu()
    assert abs(float(got[0]) - norm) <= 2.0 ** -23 * norm
    assert abs(float(got[1]) - 0.01 / (norm + 1e-6)) <= 2.0 ** -21 * float(got[1]) and float(got[1]) < 1
    for i, (t, e) in enumerate(zip(ts, opt.entries)):
        same(e, expect(t, i, bits, True, 5, 1e-3, 7, coef=float(got[1])), bits, True)


def test_norm_below_the_limit_and_at_extremes():
    for vals, want in [([0.0] * 10, 0.0), ([1e-30] * 4, 2e-30), ([1e30] * 4, 2e30), ([3.0, 4.0], 5.0)]:
        g = torch.tensor(vals, device="cuda")
        arr = A.adamw_tensors([A.adamw_tensor(len(vals), None, None, g, None, None)])
        out = torch.empty(2, device="cuda")
        ws = torch.empty(A.fp8mlp_grad_norm_workspace_size(arr), dtype=U8, device="cuda")
        A.fp8mlp_grad_norm(arr, 10.0, out, ws)
        torch.cuda.synchronize()
        assert float(out[0]) == pytest.approx(want, rel=2.0 ** -23) and float(out[1]) == pytest.approx(min(1.0, 10 / (want + 1e-6)))
    # no tensors at all; 300 of them (three launches)
    out = torch.empty(2, device="cuda")
    empty = A.adamw_tensors([])
    A.fp8mlp_grad_norm(empty, 1.0, out, torch.empty(16, dtype=U8, device="cuda"))
    assert out.tolist() == [0.0, 1.0]
    gs = [torch.full((i + 1,), 0.5, device="cuda") for i in range(300)]
    arr = A.adamw_tensors([A.adamw_tensor(g.numel(), None, None, g, None, None) for g in gs])
    ws = torch.empty(A.fp8mlp_grad_norm_workspace_size(arr), dtype=U8, device="cuda")
    A.fp8mlp_grad_norm(arr, float("inf"), out, ws)
    torch.cuda.synchronize()
    assert float(out[0]) == pytest.approx((0.25 * 300 * 301 / 2) ** 0.5, rel=2.0 ** -23) and float(out[1]) == 1.0


@pytest.mark.parametrize("sizes", [[1], [3, 4, 5], [4096, 4097, 8191, 1], [1537] * 60, [0, 5000, 0, 1], [1 << 20], [(1 << 20) + 1],
                                   [8193] * 127, [8193] * 128, [700] * 129, [0] * 200 + [9], [2359296] * 3 + [5]])
def test_norm_against_float64(sizes):
    g = torch.Generator(device="cuda").manual_seed(sum(sizes) + len(sizes))
    gs = [torch.randn(n, generator=g, device="cuda") * torch.exp(4 * torch.randn(1, generator=g, device="cuda")) for n in sizes]
    arr = A.adamw_tensors([A.adamw_tensor(x.numel(), None, None, x, None, None) for x in gs])
    out, ws = torch.empty(2, device="cuda"), torch.empty(A.fp8mlp_grad_norm_workspace_size(arr), dtype=U8, device="cuda")
    A.fp8mlp_grad_norm(arr, 0.25, out, ws)
    want = float(sum(x.double().square().sum() for x in gs)) ** 0.5
    # sums in double: the result's own rounding, one division and one sum
    assert abs(float(out[0]) - want) <= 2.0 ** -23 * want
    assert abs(float(out[1]) - min(1.0, 0.25 / (want + 1e-6))) <= 2.0 ** -21 * float(out[1])
    again = torch.empty_like(out)
    A.fp8mlp_grad_norm(arr, 0.25, again, ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_without_a_finite_norm_is_skipped(bad, bits):
    ts = tensors([300, 5000], bits, True)
    ts[1]["g"][4321] = bad
    opt, raws = build(ts, bits, True, max_norm=1.0)
    before = [r.clone() for r in raws]
    opt.step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, raws))
    assert opt.read_state()["step"] == 4 and opt.read_state()["skipped"] == 1
    assert A.fp8mlp_get_device_status() & A.STATUS_STEP_SKIPPED
    A.fp8mlp_clear_device_status()
    # and the next one is taken
    opt.entries[1]["grad"][4321] = 0.0
    opt.step()
    torch.cuda.synchronize()
    assert opt.read_state()["step"] == 5 and A.fp8mlp_get_device_status() == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_advance(bits):
    ts = tensors([700, 5000, 129], bits, False)
    a, _ = build(ts, bits, False, max_norm=1.0)
    b, _ = build(ts, bits, False, max_norm=1.0)
    for _ in range(4):
        a.step()
    b.step()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        b.step()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert a.read_state() == b.read_state() and a.read_state()["step"] == 8
    for x, y in zip(a.entries, b.entries):
        assert all(torch.equal(x[k].view(U8), y[k].view(U8)) for k in x if x[k] is not None)
    # a new rate reaches the captured step
    b.set_lr(0.0)
    before = b.entries[1]["weight"].clone()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(before, b.entries[1]["weight"])


def test_another_stream_and_two_optimizers_at_once():
    ts = tensors([20000, 333], 8, True)
    one, _ = build(ts, 8, True)
    two, _ = build(ts, 8, True)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    one.stream, two.stream = s1, s2
    for _ in range(5):
        one.step()
        two.step()
    torch.cuda.synchronize()
    for x, y in zip(one.entries, two.entries):
        assert all(torch.equal(x[k].view(U8), y[k].view(U8)) for k in x)


def test_an_optimizer_on_a_stream_of_its_own_from_the_start():
    # its buffers are zeroed on the current stream, which is kept busy here
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    g, w = torch.full((5000,), 0.5, device="cuda"), torch.zeros(5000, device="cuda")
    for _ in range(20):
        a = a @ a * 1e-3
    opt = AdamW(state_bits=8, lr=1e-2, seed=9, step_count=6, max_norm=1.0, stream=side)
    e = opt.add(g, master=w)
    for _ in range(20):
        a = a @ a * 1e-3
    opt.step()
    side.synchronize()
    s = opt.state.clone()
    torch.cuda.synchronize()
    assert opt.read_state() == dict(lr=R.f32(1e-2), step=7, seed=9, skipped=0) and torch.equal(s, opt.state)
    assert bool((w != 0).all()) and bool((e["v"].float() > 0).all())


@pytest.mark.parametrize("handle", [False, True])
def test_lr_and_state_with_a_stream_of_its_own(handle):
    a = torch.randn(4096, 4096, device="cuda")
    g, w = torch.full((3000,), 0.5, device="cuda"), torch.zeros(3000, device="cuda")
    side = torch.cuda.Stream()
    opt = AdamW(lr=1e-2, stream=side.cuda_stream if handle else side)
    opt.add(g, master=w)
    opt.step()
    side.synchronize()
    first = w.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # a step that waits behind other work
        for _ in range(20):
            a = a @ a * 1e-3
    opt.step()
    opt.set_lr(0.0)  # of the third step, not of the second
    assert opt.read_state() == dict(lr=0.0, step=2, seed=0, skipped=0)
    second = w.clone()
    torch.cuda.synchronize()
    for _ in range(20):
        a = a @ a * 1e-3
    opt.step()  # lr = 0 has arrived although the current stream is busy
    assert opt.read_state()["step"] == 3
    torch.cuda.synchronize()
    assert bool((second < first).all()) and torch.equal(w, second)


def test_state_carries_over():
    ts = tensors([999], 8, True)
    a, _ = build(ts, 8, True)
    a.step()
    saved = {k: v.clone() for k, v in a.entries[0].items()}
    st = a.state.clone()
    a.step()
    b = AdamW(state_bits=8, betas=(HYPER["b1"], HYPER["b2"]), eps=HYPER["eps"])
    b.state.copy_(st)
    b.add(saved["grad"], saved["master"], saved["weight"], weight_decay=0.1,
          state={k: saved[k] for k in ("m", "v", "m_scale", "v_scale")})
    b.step()
    torch.cuda.synchronize()
    assert all(torch.equal(a.entries[0][k].view(U8), b.entries[0][k].view(U8)) for k in saved)


def test_refusals():
    opt = AdamW()
    g, p = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    with pytest.raises(ValueError, match="master or weight"):
        opt.add(g)
    with pytest.raises(ValueError, match="size"):
        opt.add(g, master=p[:8])
    with pytest.raises(ValueError, match="fp32"):
        opt.add(g.to(BF), master=p)
    with pytest.raises(ValueError, match="bits"):
        opt.add(g, master=p, state={"m": torch.zeros(10, dtype=F8, device="cuda"), "v": torch.zeros(10, dtype=F8, device="cuda")})
    opt.add(g, master=p)
    with pytest.raises(ValueError, match="twice"):
        opt.add(torch.zeros(10, device="cuda"), master=p)
    with pytest.raises(ValueError, match="twice"):
        opt.add(p, master=p)
    with pytest.raises(ValueError, match="CUDA"):
        opt.add(torch.zeros(10), master=torch.zeros(10))


def test_offsets_beyond_32_bits():
    # one tensor of 2^31 + 300 elements, 8-bit states: its first and last elements
    n = 2 ** 31 + 300
    g = torch.full((n,), 1e-3, device="cuda")
    w = torch.full((n,), 0.5, dtype=BF, device="cuda")
    opt = AdamW(state_bits=8, lr=1e-2, seed=3)
    e = opt.add(g, weight=w, weight_decay=0.0)
    opt.step()
    torch.cuda.synchronize()
    z = torch.zeros(n % 128 + 896, device="cuda")
    for first in (0, n - z.numel()):
        c = z.numel()
        p, m, v = R.adamw(z + 0.5, z + 1e-3, z.clone(), z.clone(), 1, 1e-2, 0.0, 0.9, 0.95, 1e-8)
        r = R.random_bits(c, 0, 1, 3, first, device="cuda")
        assert torch.equal(w[first:first + c], R.bf16_stochastic(p, R.mix32(r ^ 0x5BD1E995) & 0xFFFF).to(BF))
        mq, ms = R.quant_state(m, (r & 0xFFFF).float() * 2.0 ** -16, False)
        assert torch.equal(e["m"][first:first + c].float(), mq)
        assert torch.equal(e["m_scale"][first // 128:first // 128 + ms.numel()], ms)


@pytest.mark.parametrize("handle", [False, True])
def test_parameters_added_between_steps_on_a_stream_of_its_own(handle):
    # the first step still waits when the second's larger workspace is made and other tensors take what is free
    a = torch.randn(4096, 4096, device="cuda")
    n = [20000, 16384 * 300]
    g = [torch.full((k,), 0.5 + i, device="cuda") for i, k in enumerate(n)]
    w = [torch.zeros(k, device="cuda") for k in n]
    side = torch.cuda.Stream()
    opt = AdamW(lr=1e-2, max_norm=1.0, stream=side.cuda_stream if handle else side)
    opt.add(g[0], master=w[0])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            a = a @ a * 1e-3
    opt.step()
    opt.add(g[1], master=w[1])
    opt.step()
    others = [torch.full((64,), float(i), device="cuda") for i in range(200)]
    torch.cuda.synchronize()
    assert all(bool((t == i).all()) for i, t in enumerate(others))
    assert opt.read_state()["step"] == 2

    def coef(k):  # of the first k gradients, in fp32 as the call works it out
        norm = torch.tensor(sum(n[i] * (0.5 + i) ** 2 for i in range(k)), dtype=torch.float64).sqrt().float()
        return norm, 1.0 / (norm + 1e-6)
    assert float(opt.norm[0]) == float(coef(2)[0])
    for i in range(2):
        p = m = v = torch.zeros(1)
        for t in range(1 + i, 3):
            p, m, v = R.adamw(p, torch.tensor([0.5 + i]), m, v, t, 1e-2, 0.0, 0.9, 0.95, 1e-8, coef=float(coef(t)[1]))
        assert bool((w[i].cpu() == p).all())


def test_a_first_step_captured_on_a_stream_of_its_own():
    side = torch.cuda.Stream()
    g, w = torch.full((5000,), 0.5, device="cuda"), torch.zeros(5000, device="cuda")
    opt = AdamW(lr=1e-2, max_norm=1.0, stream=side)
    opt.add(g, master=w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        opt.step()
    assert opt.read_state()["step"] == 0
    # the captured step goes on with its own parameter after another has come
    extra = torch.zeros(1 << 18, device="cuda")
    opt.add(torch.ones(1 << 18, device="cuda"), master=extra)
    opt.step()
    torch.cuda.synchronize()
    after = extra.clone()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert opt.read_state()["step"] == 4 and torch.equal(after, extra) and bool((w < -3e-2).all())
    assert float(opt.norm[0]) == pytest.approx(0.5 * 5000 ** 0.5, rel=2.0 ** -22)


@pytest.mark.parametrize("bits", [32, 8])
def test_overlapping_arrays_are_refused(bits):
    ts = tensors([300, 5000], bits, True)
    opt, raws = build(ts, bits, True, max_norm=1.0)
    before = [r.clone() for r in raws]
    norm = opt.norm.clone()
    torch.cuda.synchronize()
    arr = A.adamw_tensors(opt._descriptors)
    arr[1].p = arr[0].g + 16
    with pytest.raises(A.Fp8MlpError, match="overlaps") as e:
        A.fp8mlp_adamw_step(arr, opt.state, bits, 0.9, 0.95, 1e-8)
    assert e.value.code == A.ERR_INVALID_ARG
    ws = torch.empty(A.fp8mlp_grad_norm_workspace_size(arr), dtype=U8, device="cuda")
    with pytest.raises(A.Fp8MlpError, match="overlaps"):
        A.fp8mlp_grad_norm(arr, 1.0, opt.entries[0]["grad"], ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, raws)) and torch.equal(norm, opt.norm)
    assert opt.read_state()["step"] == 4
    opt.step()
    assert opt.read_state()["step"] == 5
