"""Host-side refusals of the block-scaled products, the gated norms and the
optimizer (no GPU needed: arguments are checked before any CUDA call), the
descriptor's layout, and the plain definitions against differences."""
import ctypes
import math
import random
import re

import pytest
import torch

from fp8_relu_mlp_b200 import _abi as A
import train_ops_ref as R

F = 0x10000  # 16-byte aligned, never dereferenced on the host
INVALID, SHAPE = A.ERR_INVALID_ARG, A.ERR_UNSUPPORTED_SHAPE


@pytest.fixture(autouse=True, params=["python", "compiled"])
def marshalling(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(A, "_marshal", None)
    elif A._marshal is None:
        monkeypatch.setattr(A, "_marshal", None)  # put back afterwards
        A._find_marshal(torch)
        if A._marshal is None:
            pytest.skip("the module is not built")


def refused(code, fn, *args):
    with pytest.raises(A.Fp8MlpError) as e:
        fn(*args, stream=0)
    assert e.value.code == code, str(e.value)


APART = [F * (i + 1) for i in range(11)]  # the largest array of these sizes has 32 KiB
BLOCK_CALLS = {
    "linear_fwd_block": (A.fp8mlp_linear_fwd_block, [4, 128, 256], APART[:5]),
    "linear_block": (A.fp8mlp_linear_block, [4, 128, 256], APART[:6]),
    "up_proj_block": (A.fp8mlp_up_proj_block, [4, 128, 256], APART[:7]),
    "mlp_fwd_block": (A.fp8mlp_mlp_fwd_block, [4, 128, 256], APART[:11]),
    "quantize_block": (A.fp8mlp_quantize_block, [4, 128], APART[:3]),
}
OUTPUTS = {"linear_fwd_block": [4], "linear_block": [3, 4, 5], "up_proj_block": [4, 5, 6], "mlp_fwd_block": [5, 6, 7, 8, 9, 10],
           "quantize_block": [1, 2]}


@pytest.mark.parametrize("name", BLOCK_CALLS)
def test_block_products_refuse(name):
    fn, sizes, ptrs = BLOCK_CALLS[name]
    refused(INVALID, fn, -1, *sizes[1:], *ptrs)
    for i in range(1, len(sizes)):
        for bad in (0, 8, 24, -16, (1 << 22) + 16):
            refused(SHAPE, fn, *[bad if k == i else v for k, v in enumerate(sizes)], *ptrs)
    for i in range(len(ptrs)):
        refused(INVALID, fn, *sizes, *[None if k == i else v for k, v in enumerate(ptrs)])
        refused(INVALID, fn, *sizes, *[F + 2 if k == i else v for k, v in enumerate(ptrs)])
    # an empty batch is no error and touches nothing
    assert fn(0, *sizes[1:], *[None] * len(ptrs), stream=0) == A.OK
    if not torch.cuda.is_available():
        refused(A.ERR_NO_DEVICE, fn, *sizes, *ptrs)


@pytest.mark.parametrize("name", BLOCK_CALLS)
def test_block_products_refuse_overlaps(name):
    fn, sizes, ptrs = BLOCK_CALLS[name]
    M, K = sizes[:2]
    N = sizes[2] if len(sizes) > 2 else 0
    size = {"linear_fwd_block": [M * K, 4 * M, N * K, 8, 2 * M * N], "linear_block": [2 * M * K, N * K, 8, M * K, 4 * M, 2 * M * N],
            "up_proj_block": [M * K, 4 * M, N * K, 8, 2 * M * N, M * N, 8 * M], "quantize_block": [2 * M * K, M * K, 4 * M],
            "mlp_fwd_block": [2 * M * K, N * K, 8, N * K, 8, M * K, 4 * M, 2 * M * N, M * N, 8 * M, 2 * M * K]}[name]
    for o in OUTPUTS[name]:
        for i in range(len(ptrs)):
            if i == o or (name == "mlp_fwd_block" and {i, o} == {0, 10}):
                continue
            for at in (ptrs[i], ptrs[i] + (size[i] - 1) // 16 * 16, ptrs[i] - (size[o] - 1) // 16 * 16):
                refused(INVALID, fn, *sizes, *[at if k == o else v for k, v in enumerate(ptrs)])
            if not torch.cuda.is_available():  # side by side is no overlap
                for at in (ptrs[i] + -(-size[i] // 16) * 16, ptrs[i] - -(-size[o] // 16) * 16):
                    refused(A.ERR_NO_DEVICE, fn, *sizes, *[at if k == o else v for k, v in enumerate(ptrs)])
    if name == "mlp_fwd_block" and not torch.cuda.is_available():
        refused(A.ERR_NO_DEVICE, fn, *sizes, *ptrs[:-1], ptrs[0])


def test_weight_cache_refuses():
    f = A.fp8mlp_weight_block_cache_refresh
    refused(SHAPE, f, 24, 16, F, F, F, F, F)
    refused(SHAPE, f, (1 << 22) + 16, 16, F, F, F, F, F)
    refused(INVALID, f, 16, 16, None, F, F, F, F)
    refused(INVALID, f, 16, 16, F, None, None, None, None)
    refused(INVALID, f, 16, 16, F, F, None, None, None)
    refused(INVALID, f, 16, 16, F, F, F, F, None)
    refused(INVALID, f, 16, 16, F, F + 8, F, None, None)
    far = [F * k for k in range(1, 6)]
    for o in range(1, 5):
        for i in range(5):
            if i != o:
                refused(INVALID, f, 16, 16, *[far[i] if k == o else v for k, v in enumerate(far)])


FWD = dict(M=4, d=64, r=F, y=F, w_post=F, gate=F, rows_per_gate=2, alpha=F, w_pre=F, eps=1e-6, r_next=F, rstd_post=F, x=F,
           rstd_pre=F, xq=F, xs=F)
BWD = dict(M=4, d=64, r=F, y=F, w_post=F, gate=F, rows_per_gate=2, alpha=F, rstd_post=F, r_next=F, w_pre=F, rstd_pre=F, dx=F,
           dr_next=F, dr=F, dy=F, dw_post=F, dgate=F, dalpha=F, dw_pre=F, workspace=F)


@pytest.mark.parametrize("code,change", [
    (INVALID, dict(M=-1)), (SHAPE, dict(d=24)), (SHAPE, dict(d=8208)), (INVALID, dict(rows_per_gate=0)),
    (INVALID, dict(eps=0.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))), (INVALID, dict(r=None)),
    (INVALID, dict(xq=None)), (INVALID, dict(xs=None)), (INVALID, dict(r_next=None)), (INVALID, dict(rstd_post=None)),
    (INVALID, dict(rstd_pre=None)), (INVALID, dict(y=None)), (INVALID, dict(x=None)), (INVALID, dict(r=F + 8)),
    (INVALID, dict(gate=F + 4)), (INVALID, dict(alpha=F + 2)), (INVALID, dict(xq=F + 4)), (INVALID, dict(w_pre=F + 2)),
    (INVALID, dict(y=None, w_post=None, gate=None, alpha=None, r_next=None, rstd_post=None, x=None, w_pre=None,
                   rstd_pre=None, xq=None, xs=None))])
def test_norms_refuse(code, change):
    refused(code, A.fp8mlp_norm_gate_fwd, *dict(FWD, **change).values())


@pytest.mark.parametrize("code,change", [
    (INVALID, dict(M=-1)), (SHAPE, dict(d=8)), (SHAPE, dict(d=8208)), (INVALID, dict(rows_per_gate=-3)),
    (INVALID, dict(r=None)), (INVALID, dict(y=None)), (INVALID, dict(dx=None)), (INVALID, dict(dr=None)),
    (INVALID, dict(dy=None)), (INVALID, dict(rstd_post=None)), (INVALID, dict(rstd_pre=None)), (INVALID, dict(r_next=None)),
    (INVALID, dict(workspace=None)), (INVALID, dict(workspace=F + 8)), (INVALID, dict(dgate=F + 4)),
    (INVALID, dict(dr_next=F + 2)), (INVALID, dict(dalpha=F + 1))])
def test_norm_gradients_refuse(code, change):
    refused(code, A.fp8mlp_norm_gate_bwd, *dict(BWD, **change).values())


@pytest.mark.parametrize("M,d,rows", [(1, 16, 1), (16384, 768, 16384), (5000, 1040, 7), (3, 8192, 1)])
def test_norm_workspace_covers_the_parts(M, d, rows):
    need = A.fp8mlp_norm_gate_bwd_workspace_size(M, d, rows)
    assert need >= 2 * 4 * d + 8 and need <= 8 * 4 * d * 2400
    assert A.fp8mlp_norm_gate_bwd_workspace_size(0, d, rows) == 0
    assert A.fp8mlp_norm_gate_bwd_workspace_size(M, d, 0) == 0


def tensor(**kw):
    d = dict(n=10, p=F, p_bf16=F, g=F, m=F, v=F, m_scale=F, v_scale=F, lr_mult=1.0, weight_decay=0.0)
    return A.adamw_tensors([A.AdamwTensor(*dict(d, **kw).values())])


@pytest.mark.parametrize("code,change", [
    (INVALID, dict(n=-1)), (SHAPE, dict(n=(1 << 42) + 1)), (SHAPE, dict(n=1 << 42, )), (INVALID, dict(g=None)),
    (INVALID, dict(g=F + 4)), (INVALID, dict(p=None, p_bf16=None)), (INVALID, dict(p=F + 8)), (INVALID, dict(p_bf16=F + 2)),
    (INVALID, dict(m=None)), (INVALID, dict(v=None)), (INVALID, dict(m_scale=None)), (INVALID, dict(v_scale=F + 1)),
    (INVALID, dict(lr_mult=float("nan"))), (INVALID, dict(weight_decay=float("inf")))])
def test_adamw_refuses_tensors(code, change):
    if change == dict(n=1 << 42):
        arr = A.adamw_tensors([tensor(**change)[0], tensor(**change)[0], tensor(n=1 << 41)[0]] + [tensor(**change)[0]] * 2)
    else:
        arr = tensor(**change)
    refused(code, A.fp8mlp_adamw_step, arr, F, 8, 0.9, 0.95, 1e-8, F)


@pytest.mark.parametrize("args", [(F, 16, 0.9, 0.95, 1e-8, None), (None, 8, 0.9, 0.95, 1e-8, None),
                                  (F, 8, 1.0, 0.95, 1e-8, None), (F, 8, 0.9, -0.1, 1e-8, None),
                                  (F, 8, 0.9, float("nan"), 1e-8, None), (F, 8, 0.9, 0.95, 0.0, None),
                                  (F, 8, 0.9, 0.95, 1e-8, F + 2), (F + 8, 8, 0.9, 0.95, 1e-8, None)])
def test_adamw_refuses_scalars(args):
    refused(INVALID, A.fp8mlp_adamw_step, tensor(), *args)


def test_optimizer_helpers_refuse():
    refused(INVALID, A.fp8mlp_grad_norm, tensor(), 0.0, F, F)
    refused(INVALID, A.fp8mlp_grad_norm, tensor(), float("nan"), F, F)
    refused(INVALID, A.fp8mlp_grad_norm, tensor(), 1.0, None, F)
    refused(INVALID, A.fp8mlp_grad_norm, tensor(), 1.0, F, None)
    refused(INVALID, A.fp8mlp_grad_norm, tensor(n=-2), 1.0, F, F)
    refused(INVALID, A.fp8mlp_adamw_state_init, F, float("inf"), 0, 0)
    refused(INVALID, A.fp8mlp_adamw_state_init, F, 1e-3, 0, -1)
    with pytest.raises(TypeError):
        A.fp8mlp_adamw_step([], F, 8, 0.9, 0.95, 1e-8)
    with pytest.raises(ValueError, match="CUDA"):
        A.adamw_tensor(4, torch.zeros(4), None, torch.zeros(4), torch.zeros(4), torch.zeros(4))
    # scales are not asked for with 32-bit states
    if not torch.cuda.is_available():
        refused(A.ERR_NO_DEVICE, A.fp8mlp_adamw_step, tensor(m_scale=None, v_scale=None), F, 32, 0.9, 0.95, 1e-8, None)
    assert A.fp8mlp_grad_norm_workspace_size(tensor(n=16385)) == 16
    assert A.fp8mlp_grad_norm_workspace_size(A.adamw_tensors([])) == 16
    assert A.fp8mlp_grad_norm_workspace_size(tensor(n=16384 * 5 + 1)) == 48


def test_struct_layouts():
    text = open(A.HEADER).read()
    body = re.search(r"typedef struct fp8mlp_adamw_state \{(.*?)\} fp8mlp_adamw_state;", text, re.S).group(1)
    fields = re.findall(r"(?:float|int32_t|uint32_t)\s+\w+(?:\[(\d+)\])?;", body)
    assert sum(4 * int(f or 1) for f in fields) == 32
    body = re.search(r"typedef struct fp8mlp_adamw_tensor \{(.*?)\} fp8mlp_adamw_tensor;", text, re.S).group(1)
    names = re.findall(r"(\w+);", body)
    assert names == [f[0] for f in A.AdamwTensor._fields_] and ctypes.sizeof(A.AdamwTensor) == 72


def test_the_plain_norm_gradient_agrees_with_differences():
    torch.manual_seed(0)
    M, d, rows = 7, 32, 3
    t = lambda *s: torch.randn(*s, dtype=R.F64)  # noqa: E731
    q = dict(r=t(M, d), y=t(M, d), w_post=t(d), gate=t(3, d), alpha=t(1), w_pre=t(d))
    cx, cr = t(M, d), t(M, d)

    def loss(q):
        rn, _, x, _ = R.norms_fwd(q["r"], q["y"], q["w_post"], q["gate"], rows, q["alpha"], q["w_pre"], 1e-6)
        return float((x * cx).sum() + (rn * cr).sum())

    rn, rpost, _, rpre = R.norms_fwd(q["r"], q["y"], q["w_post"], q["gate"], rows, q["alpha"], q["w_pre"], 1e-6)
    out, _ = R.norms_bwd(q["r"], q["y"], q["w_post"], q["gate"], rows, q["alpha"], rpost, rn, q["w_pre"], rpre, cx, cr)
    for k, g in dict(r="dr", y="dy", w_post="dw_post", gate="dgate", alpha="dalpha", w_pre="dw_pre").items():
        v = torch.randn_like(q[k])
        num = (loss({**q, k: q[k] + 1e-6 * v}) - loss({**q, k: q[k] - 1e-6 * v})) / 2e-6
        assert abs(num - float((out[g] * v).sum())) < 1e-5 * (1 + abs(num)), k


def test_the_plain_step_agrees_with_float64():
    torch.manual_seed(1)
    n = 500
    p, g, m, v = torch.randn(n) * 0.02, torch.randn(n) * 1e-3, torch.randn(n) * 1e-3, torch.rand(n) * 1e-6
    a = R.adamw(p, g, m, v, 7, 1e-3, 0.1, 0.9, 0.95, 1e-8)
    b = R.adamw64(p, g, m, v, 7, 1e-3, 0.1, 0.9, 0.95, 1e-8)
    for x, y in zip(a, b):
        assert float((x.double() - y).abs().max()) <= 2.0 ** -20 * float(y.abs().max())


def test_stochastic_rounding_of_the_plain_form():
    # between two codes with the right frequency, never beyond them, exact codes kept
    n = 1 << 16
    u = torch.arange(n).float() / n
    for x, lo, hi in [(100.0, 96.0, 104.0), (1.03, 1.0, 1.125), (0.003, 2.0 ** -9, 2.0 ** -8), (448.0, 448.0, 448.0)]:
        t = torch.full((n,), x)
        t[::128] = 448.0  # every block's scale is 1
        q, s = R.quant_state(t, u, False)
        assert bool((s == 1).all())
        rest = q[torch.arange(n) % 128 != 0]
        assert set(rest.tolist()) <= {lo, hi} and abs(float(rest.mean()) - x) < 1e-3 * x + 2e-5


# the norms' arrays apart from each other, their sizes, which ones are written, and the pairs that may be one array
NORM_SIZES = dict(r=512, y=512, w_post=128, gate=256, alpha=4, w_pre=128, r_next=512, rstd_post=16, x=512, rstd_pre=16, xq=256,
                  xs=16, dx=512, dr_next=512, dr=512, dy=512, dw_post=256, dgate=512, dalpha=4, dw_pre=256)
NORM_CALLS = {
    "fwd": (A.fp8mlp_norm_gate_fwd, FWD, ["r_next", "rstd_post", "x", "rstd_pre", "xq", "xs"], [("r_next", "r"), ("x", "y")]),
    "bwd": (A.fp8mlp_norm_gate_bwd, BWD, ["dr", "dy", "dw_post", "dgate", "dalpha", "dw_pre", "workspace"],
            [("dr", "dr_next"), ("dy", "y"), ("dy", "dx")])}


@pytest.mark.parametrize("name", NORM_CALLS)
def test_norms_refuse_overlaps(name):
    fn, base, outputs, in_place = NORM_CALLS[name]
    arrays = [k for k, v in base.items() if v == F]
    far = 1 << 24
    args = dict(base, **{k: far * (i + 1) for i, k in enumerate(arrays)})
    size = dict(NORM_SIZES, workspace=A.fp8mlp_norm_gate_bwd_workspace_size(4, 64, 2))
    cpu = not torch.cuda.is_available()  # a call that is in order would run
    if cpu:
        refused(A.ERR_NO_DEVICE, fn, *args.values())
    for o in outputs:
        for i in arrays:
            if i == o:
                continue
            # the same place, all but the last 16 bytes apart, and side by side
            for at in (args[i], args[i] + (size[i] - 1) // 16 * 16, args[i] - (size[o] - 1) // 16 * 16):
                if at == args[i] and (o, i) in in_place:
                    if cpu:
                        refused(A.ERR_NO_DEVICE, fn, *{**args, o: at}.values())
                else:
                    refused(INVALID, fn, *{**args, o: at}.values())
            if cpu:
                for at in (args[i] + -(-size[i] // 16) * 16, args[i] - -(-size[o] // 16) * 16):
                    refused(A.ERR_NO_DEVICE, fn, *{**args, o: at}.values())
    for o, i in in_place:  # an array worked on in place is an output towards the others
        for k in arrays:
            if k != o and (o, k) not in in_place:
                refused(INVALID, fn, *{**args, o: args[i], k: args[i]}.values())


def test_norms_leave_unread_arrays_alone():
    if torch.cuda.is_available():
        pytest.skip("the calls would run")
    args = dict(BWD, **{k: (i + 1) << 24 for i, k in enumerate(k for k, v in BWD.items() if v == F)})
    # r is read for dalpha alone, r_next for dx
    refused(A.ERR_NO_DEVICE, A.fp8mlp_norm_gate_bwd, *{**args, "dalpha": None, "r": args["dr"]}.values())
    no_x = dict(dx=None, w_pre=None, rstd_pre=None, dw_pre=None)
    refused(A.ERR_NO_DEVICE, A.fp8mlp_norm_gate_bwd, *{**args, **no_x, "r_next": args["dr"]}.values())
    refused(INVALID, A.fp8mlp_norm_gate_bwd, *{**args, **no_x, "r": args["dr"]}.values())
    no_y = dict(y=None, w_post=None, gate=None, alpha=None, rstd_post=None, dy=None, dw_post=None, dgate=None, dalpha=None)
    refused(A.ERR_NO_DEVICE, A.fp8mlp_norm_gate_bwd, *{**args, **no_y}.values())
    refused(INVALID, A.fp8mlp_norm_gate_bwd, *{**args, **no_y, "r_next": args["dr"]}.values())


def descriptors(n=3, size=1000, flat=True, order=None):
    """Tensors of ``size`` elements with arrays apart, as in flat buffers or one after another."""
    names = ["p", "p_bf16", "g", "m", "v", "m_scale", "v_scale"]
    out = []
    for i in range(n) if order is None else order:
        at = {k: ((j + 1) << 28) + (i << 16) if flat else ((i + 1) << 28) + (j << 16) for j, k in enumerate(names)}
        out.append(dict(n=size, **at))
    return out


def adamw_array(ts):
    return A.adamw_tensors([A.AdamwTensor(lr_mult=1.0, weight_decay=0.0, **t) for t in ts])


ST, COEF = 1 << 40, (1 << 40) + 32


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("flat,order", [(True, None), (False, None), (True, [2, 0, 1]), (False, [1, 2, 0])])
def test_adamw_refuses_overlaps(bits, flat, order):
    def check(code, ts, st=ST, coef=COEF):
        if code == A.OK:
            assert A.fp8mlp_adamw_check(adamw_array(ts), st, bits, coef) == A.OK
        else:
            with pytest.raises(A.Fp8MlpError, match="overlaps") as e:
                A.fp8mlp_adamw_check(adamw_array(ts), st, bits, coef)
            assert e.value.code == code

    def make():
        return descriptors(3, 1000, flat, order)
    check(A.OK, make())
    check(A.OK, make(), coef=None)
    size = dict(p=4000, p_bf16=2000, g=4000, m=1000 * bits // 8, v=1000 * bits // 8, m_scale=32, v_scale=32)
    scales = ("m_scale", "v_scale")
    for i in range(3):
        for k in size:
            for j in range(3):
                for q in size:
                    if (i, k) == (j, q):
                        continue
                    unread = bits == 32 and (k in scales or q in scales)
                    harmless = unread or (k == "g" and q == "g")  # nothing is written there
                    for shift in (0, (size[q] - 1) // 16 * 16, -((size[k] - 1) // 16 * 16)):
                        ts = make()
                        ts[i][k] = ts[j][q] + shift
                        check(A.OK if harmless else INVALID, ts)
                    for shift in (-(-size[q] // 16) * 16, -(-(-size[k] // 16) * 16)):  # side by side
                        ts = make()
                        ts[i][k] = ts[j][q] + shift
                        check(A.OK, ts)
            unread = bits == 32 and k in scales
            ts = make()
            ts[i][k] = ST
            check(A.OK if unread else INVALID, ts)
            ts[i][k] = COEF - 16
            check(A.OK if unread else INVALID, ts)
            ts[i][k] = COEF
            check(A.OK if unread or k == "g" else INVALID, ts)
    check(INVALID, make(), coef=ST + 8)
    # empty tensors have no arrays
    ts = make()
    ts[1].update(n=0, p=ts[0]["p"], g=ts[0]["p"])
    check(A.OK, ts)
    ts[1].update(n=1)
    check(INVALID, ts)


def test_many_overlapping_arrays_are_found():
    ts = descriptors(300, 1000)
    assert A.fp8mlp_adamw_check(adamw_array(ts), ST, 8, COEF) == A.OK
    ts.reverse()
    assert A.fp8mlp_adamw_check(adamw_array(ts), ST, 8, COEF) == A.OK
    # a gradient that spans others' (fine) and, behind them, a weight
    ts[7]["n"] = 1000000
    ts[7].update(g=1 << 50, p=(1 << 50) + (1 << 30), p_bf16=(1 << 51), m=1 << 52, v=1 << 53, m_scale=1 << 54, v_scale=1 << 55)
    ts[8]["g"], ts[9]["g"], ts[10]["g"] = (1 << 50) + 16, (1 << 50) + 32, (1 << 50) + (1 << 20)
    assert A.fp8mlp_adamw_check(adamw_array(ts), ST, 8, COEF) == A.OK
    ts[11]["p"] = (1 << 50) + 3999984
    with pytest.raises(A.Fp8MlpError, match="p of tensor 11 overlaps g of tensor 7"):
        A.fp8mlp_adamw_check(adamw_array(ts), ST, 8, COEF)


def test_adamw_check_refuses_what_the_step_refuses():
    for t, st, bits in ((tensor(n=-1), F, 8), (tensor(m=None), F, 8), (tensor(), F, 16), (tensor(), None, 8), (tensor(), F + 8, 8)):
        with pytest.raises(A.Fp8MlpError) as e:
            A.fp8mlp_adamw_check(t, st, bits)
        assert e.value.code == INVALID
    assert A.fp8mlp_adamw_check(A.adamw_tensors([]), F, 8) == A.OK


def test_gradient_norm_refuses_overlaps():
    arr = adamw_array([dict(n=40000, g=1 << 20), dict(n=100, g=1 << 24), dict(n=0, g=1 << 28)])
    out, ws = 1 << 28, 1 << 29
    for bad in (dict(o=1 << 20), dict(o=(1 << 24) + 396), dict(w=(1 << 20) + 159984), dict(w=(1 << 20) - 16), dict(o=1 << 29)):
        refused(INVALID, A.fp8mlp_grad_norm, arr, 1.0, bad.get("o", out), bad.get("w", ws))
    if not torch.cuda.is_available():
        refused(A.ERR_NO_DEVICE, A.fp8mlp_grad_norm, arr, 1.0, out, ws)
        refused(A.ERR_NO_DEVICE, A.fp8mlp_grad_norm, arr, 1.0, (1 << 24) + 400, (1 << 20) - 48)


def test_norm_workspace_stays_small():
    # parts of gate rows: at most two to three times a tensor of the call, and what 148 SMs' workers take at least
    rng = random.Random(5)
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    cases = [(65536, 32, 8), (16384, 64, 8), (1000000, 64, 33), (72600000, 16, 33), (16384, 64, 9472), (20005, 16, 2)]
    for _ in range(20000):
        M, d = log(1, 5e6), 16 * log(1, 512)
        cases.append((M, d, log(1, M + 1)))
    for M, d, rows in cases:
        need = A.fp8mlp_norm_gate_bwd_workspace_size(M, d, rows)
        assert need <= 2.5 * (2 * M * d) + (16 << 20), (M, d, rows, need)


@pytest.mark.parametrize("M", [2 ** 31 - 4095, 2 ** 31 - 256, 2 ** 31 - 1])
def test_rows_next_to_2_31_are_refused(M):
    for name, (fn, sizes, ptrs) in BLOCK_CALLS.items():
        refused(SHAPE, fn, M, *[16] * (len(sizes) - 1), *ptrs)
    refused(SHAPE, A.fp8mlp_norm_gate_fwd, *dict(FWD, M=M, d=16, rows_per_gate=M).values())
    refused(SHAPE, A.fp8mlp_norm_gate_bwd, *dict(BWD, M=M, d=16, rows_per_gate=M).values())
    assert A.fp8mlp_norm_gate_bwd_workspace_size(M, 16, M) == 0


@pytest.mark.parametrize("rows", [1, 2, 33, 1000, 2 ** 30, 2 ** 31 - 4097, 2 ** 31 - 4096, 2 ** 31 - 1])
def test_the_most_rows(rows):
    M = 2 ** 31 - 4096
    need = A.fp8mlp_norm_gate_bwd_workspace_size(M, 16, rows)
    assert 0 < need <= 4.5 * M * 16  # a part per row at most, and a bit
    if not torch.cuda.is_available():
        far = lambda d: dict(d, **{k: (i + 1) << 44 for i, k in enumerate(k for k, v in d.items() if v == F)})  # noqa: E731
        refused(A.ERR_NO_DEVICE, A.fp8mlp_norm_gate_bwd, *dict(far(BWD), M=M, d=16, rows_per_gate=rows).values())
        refused(A.ERR_NO_DEVICE, A.fp8mlp_norm_gate_fwd, *dict(far(FWD), M=M, d=16, rows_per_gate=rows).values())
        for name, (fn, sizes, ptrs) in BLOCK_CALLS.items():
            refused(A.ERR_NO_DEVICE, fn, M, *[16] * (len(sizes) - 1), *[(i + 1) << 44 for i in range(len(ptrs))])


def test_descriptors_of_other_state_bits_are_refused():
    at = lambda i: (i + 1) << 24  # noqa: E731
    made = {b: A.adamw_tensor(1000, at(0), None, at(1), at(2), at(3), at(4), at(5), state_bits=b) for b in (8, 32)}
    for have, asked in ((8, 32), (32, 8)):
        for ts in ([made[have]], [made[asked], made[have]]):
            with pytest.raises(ValueError, match=f"{have}-bit"):
                A.fp8mlp_adamw_step(A.adamw_tensors(ts), ST, asked, 0.9, 0.95, 1e-8, stream=0)
    if not torch.cuda.is_available():
        for b in (8, 32):
            refused(A.ERR_NO_DEVICE, A.fp8mlp_adamw_step, A.adamw_tensors([made[b]]), ST, b, 0.9, 0.95, 1e-8, None)
    # gradients alone, for the norm, have no states
    A.adamw_tensors([A.adamw_tensor(10, None, None, at(0), None, None), made[8]])
