"""Norms with gate and residual scale, forward and gradient, against the
formulas in float64."""
import pytest
import torch

from fp8_relu_mlp_b200 import _abi as A
from gpu_util import Guarded
import train_ops_ref as R

pytestmark = pytest.mark.gpu
BF, U8, F32, F64 = torch.bfloat16, torch.uint8, torch.float32, torch.float64
EPS = 1e-6
# fp32 work on a row: sums whose longest chain is under 128 terms, and some ten products
ROW = 2.0 ** -16
HALF = 2.0 ** -8  # half a BF16 step


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(seed, *shape, scale=1.0, add=0.0, dtype=BF):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * scale + add).to(dtype)


def inputs(M, d, rows, seed=0):
    G = R.cdiv(M, rows)
    return dict(r=randn(seed, M, d, scale=2.0), y=randn(seed + 1, M, d, scale=0.3), w_post=randn(seed + 2, d, scale=0.2, add=1),
                gate=randn(seed + 3, G, d, scale=0.3, add=0.5), alpha=randn(seed + 4, 1, scale=0.1, add=0.9, dtype=F32),
                w_pre=randn(seed + 5, d, scale=0.2, add=1))


def d64(t):
    return None if t is None else t.to(F64)


def fwd(p, M, d, rows, post=True, pre=True, quant=False, stream=None, eps=EPS):
    """Guarded outputs of one call; `p` may lack parameters."""
    o = {}
    if post:
        o.update(r_next=Guarded((M, d), BF), rstd_post=Guarded((M,), F32))
    if pre:
        o.update(x=Guarded((M, d), BF), rstd_pre=Guarded((M,), F32))
    if quant:
        o.update(xq=Guarded((M, d), U8), xs=Guarded((R.cdiv(d, 128), M), F32))
    t = {k: v.t for k, v in o.items()}
    A.fp8mlp_norm_gate_fwd(M, d, p["r"], p.get("y") if post else None, p.get("w_post") if post else None,
                           p.get("gate") if post else None, rows, p.get("alpha") if post else None,
                           p.get("w_pre") if pre else None, eps, t.get("r_next"), t.get("rstd_post"), t.get("x"),
                           t.get("rstd_pre"), t.get("xq"), t.get("xs"), stream=stream)
    torch.cuda.synchronize()
    assert all(v.intact() for v in o.values())
    return t


def close(got, want, rel, mag=None):
    got, want = got.to(F64), want.to(F64)
    return bool(((got - want).abs() <= rel * want.abs() + ROW * (want.abs() if mag is None else mag) + 1e-38).all())


# widths of each variant: one warp with 1..4 vectors a lane, a CTA with 1, 2, 4; odd rows
SHAPES = [(1, 16, 1), (1, 768, 1), (5, 32, 2), (33, 256, 33), (7, 272, 3), (100, 512, 1), (19, 528, 7), (301, 768, 301),
          (64, 784, 100), (65, 1024, 64), (17, 1040, 5), (40, 2048, 40), (9, 2064, 4), (6, 4096, 1), (5, 4112, 2), (3, 8192, 3)]


# more rows than workers, so that each walks several, at every way of dealing rows out
LONG = [(20000, 48, 20000), (40001, 32, 1), (20000, 64, 7), (9000, 128, 500), (6001, 256, 6001), (4000, 512, 1), (6000, 768, 100),
        (3001, 1024, 9), (3000, 1040, 3000), (2000, 2064, 50), (1500, 4112, 1500), (700, 8192, 3)]


@pytest.mark.parametrize("M,d,rows", SHAPES + LONG)
def test_forward(M, d, rows):
    p = inputs(M, d, rows, seed=M + d)
    got = fwd(p, M, d, rows, quant=True)
    rn, rpost, x, rpre = R.norms_fwd(*(d64(p[k]) for k in ("r", "y", "w_post", "gate")), rows, d64(p["alpha"]),
                                     d64(p["w_pre"]), EPS)
    mag = (p["alpha"].to(F64) * p["r"].to(F64)).abs() + (rn - p["alpha"].to(F64) * p["r"].to(F64)).abs()
    assert close(got["rstd_post"], rpost, 0) and close(got["rstd_pre"], rpre, 0)
    assert close(got["r_next"], rn, HALF, mag)
    xmag = mag * (rpre[:, None] * p["w_pre"].to(F64)).abs()
    assert close(got["x"], x, HALF, xmag)
    # the copy: scale from the exact maximum, codes within half a step of x
    kb = R.cdiv(d, 128)
    pad = torch.zeros(M, kb * 128, dtype=F64, device="cuda")
    pad[:, :d] = x.abs()
    magp = torch.zeros_like(pad)
    magp[:, :d] = xmag
    top = pad.view(M, kb, 128).amax(2).t()
    slack = ROW * magp.view(M, kb, 128).amax(2).t()
    assert bool(((got["xs"].to(F64) * 448 - top).abs() <= slack + 2.0 ** -22 * top).all())
    val = R.row_values(got["xq"].view(torch.float8_e4m3fn), got["xs"])
    step = got["xs"].to(F64).t().repeat_interleave(128, dim=1)[:, :d] * 2.0 ** -10
    assert bool(((val - x).abs() <= 2.0 ** -4 * x.abs() + step + 2 * ROW * xmag).all())


@pytest.mark.parametrize("drop", [("w_post",), ("gate",), ("alpha",), ("w_pre",), ("w_post", "gate", "alpha", "w_pre")])
def test_parameters_left_out_are_ones(drop):
    M, d, rows = 21, 400, 4
    p = inputs(M, d, rows)
    full = dict(p)
    for k in drop:
        full[k] = torch.ones_like(p[k])
    a = fwd({k: v for k, v in p.items() if k not in drop}, M, d, rows)
    b = fwd(full, M, d, rows)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("M,d", [(9, 256), (4, 1536)])
def test_one_part_alone(M, d):
    p = inputs(M, d, M)
    both = fwd(p, M, d, M)
    only = fwd(p, M, d, M, pre=False)
    assert torch.equal(only["r_next"], both["r_next"]) and torch.equal(only["rstd_post"], both["rstd_post"])
    pre = fwd(p, M, d, M, post=False, quant=True)
    rn, _, x, rpre = R.norms_fwd(d64(p["r"]), None, None, None, 1, None, d64(p["w_pre"]), EPS)
    assert close(pre["rstd_pre"], rpre, 0) and close(pre["x"], x, HALF)
    # without gains the pre part is the stack's plain norm
    plain = fwd({"r": p["r"]}, M, d, M, post=False)
    x0, s0 = torch.empty(M, d, dtype=BF, device="cuda"), torch.empty(M, device="cuda")
    A.fp8mlp_rmsnorm_fwd(M, d, p["r"], x0, s0)
    torch.cuda.synchronize()
    assert close(plain["rstd_pre"], s0, 0) and close(plain["x"], x0, 2 * HALF)


def test_zero_rows_infinities_and_nan_stay_in_their_row():
    M, d = 6, 768
    p = inputs(M, d, M)
    p["r"][0], p["y"][0] = 0, 0
    p["y"][2, 5] = float("inf")
    p["r"][3, 7] = float("nan")
    got = fwd(p, M, d, M, quant=True)
    assert not got["x"][0].any() and not got["r_next"][0].any() and bool((got["xs"][:, 0] == 1).all())
    assert not got["xq"][0].view(torch.float8_e4m3fn).float().any()
    assert torch.isnan(got["xs"][:, 3]).all() and torch.isnan(got["x"][3]).all()
    assert torch.isnan(got["x"][2]).any()
    for m in (1, 4, 5):
        assert all(torch.isfinite(got[k][m].float()).all() for k in ("x", "r_next")) and torch.isfinite(got["xs"][:, m]).all()


def test_in_place():
    M, d = 50, 768
    p = inputs(M, d, 7)
    want = fwd(p, M, d, 7)
    r, y = p["r"].clone(), p["y"].clone()
    s1, s2 = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    A.fp8mlp_norm_gate_fwd(M, d, r, y, p["w_post"], p["gate"], 7, p["alpha"], p["w_pre"], EPS, r, s1, y, s2)
    torch.cuda.synchronize()
    assert torch.equal(r, want["r_next"]) and torch.equal(y, want["x"]) and torch.equal(s2, want["rstd_pre"])


NAMES = ("dr", "dy", "dw_post", "dgate", "dalpha", "dw_pre")


def bwd(p, s, M, d, rows, post=True, pre=True, drn=True, skip=(), stream=None):
    G = R.cdiv(M, rows)
    shapes = {"dr": ((M, d), BF), "dy": ((M, d), BF), "dw_post": ((d,), F32), "dgate": ((G, d), F32), "dalpha": ((1,), F32),
              "dw_pre": ((d,), F32)}
    names = [n for n in NAMES if n not in skip and (post or n in ("dr", "dw_pre")) and (pre or n != "dw_pre")]
    o = {n: Guarded(*shapes[n]) for n in names}
    t = {n: v.t for n, v in o.items()}
    need = A.fp8mlp_norm_gate_bwd_workspace_size(M, d, rows)
    ws = Guarded((need,), U8, fill=0xFF)
    A.fp8mlp_norm_gate_bwd(M, d, p["r"], p["y"] if post else None, p.get("w_post") if post else None,
                           p.get("gate") if post else None, rows, p.get("alpha") if post else None,
                           s["rpost"] if post else None, s["rn"] if pre else None, p.get("w_pre") if pre else None,
                           s["rpre"] if pre else None, s["dx"] if pre else None, s["drn"] if drn else None, t["dr"],
                           t.get("dy"), t.get("dw_post"), t.get("dgate"), t.get("dalpha"), t.get("dw_pre"), ws.t,
                           stream=stream)
    torch.cuda.synchronize()
    assert all(v.intact() for v in o.values()) and ws.intact()
    return t


def saved(p, M, d, rows, seed=77):
    f = fwd(p, M, d, rows)
    return dict(rn=f["r_next"], rpost=f["rstd_post"], rpre=f["rstd_pre"], dx=randn(seed, M, d, scale=1e-3),
                drn=randn(seed + 1, M, d, scale=1e-3))


def check(got, p, s, M, rows, post=True, pre=True, drn=True):
    want, mag = R.norms_bwd(d64(p["r"]), d64(p["y"]) if post else None, d64(p.get("w_post")), d64(p.get("gate")), rows,
                            d64(p.get("alpha")) if post else None, d64(s["rpost"]), d64(s["rn"]), d64(p.get("w_pre")),
                            d64(s["rpre"]), d64(s["dx"]) if pre else None, d64(s["drn"]) if drn else None)
    # sums over rows: a worker's rows one after another, then the workers' parts, 32 interleaved
    chain = (M / 592 + 592 * 2 / 32 + 64) * 2.0 ** -24 + ROW
    for k, v in got.items():
        rel = HALF if k in ("dr", "dy") else 0
        bound = rel * want[k].abs() + (ROW if k in ("dr", "dy") else chain) * 2 * mag[k] + 1e-38
        assert bool(((v.to(F64) - want[k]).abs() <= bound).all()), k


@pytest.mark.parametrize("M,d,rows", SHAPES + [(2500, 768, 2500), (3000, 256, 700), (1300, 768, 1), (2000, 1040, 2000),
                                               (1500, 16, 10), (1201, 512, 1200)] + LONG + [
    # gate rows dealt whole; shared by few and many workers; more of them than one CTA column each; runs that touch several
    (30001, 768, 20), (3000, 768, 40), (16001, 256, 33), (5000, 1024, 101), (2500, 2064, 33), (9000, 64, 2999),
    (1200, 768, 1199), (16, 768, 4), (17, 768, 4), (13, 400, 13)])
def test_gradient_against_the_formula(M, d, rows):
    p = inputs(M, d, rows, seed=M + d)
    s = saved(p, M, d, rows)
    check(bwd(p, s, M, d, rows), p, s, M, rows)


@pytest.mark.parametrize("case", [dict(drn=False), dict(post=False), dict(pre=False), dict(skip=("dw_post", "dgate")),
                                  dict(skip=("dalpha", "dw_pre"))])
@pytest.mark.parametrize("d", [768, 1040])
def test_gradient_with_parts_left_out(case, d):
    M, rows = 130, 40
    p = inputs(M, d, rows)
    s = saved(p, M, d, rows)
    if case.get("post", True) is False:
        s = dict(s, rn=p["r"], rpre=fwd(p, M, d, rows, post=False)["rstd_pre"])
    got = bwd(p, s, M, d, rows, **case)
    check(got, p, s, M, rows, **{k: v for k, v in case.items() if k != "skip"})
    for drop in (("w_post",), ("gate",), ("alpha",), ("w_pre",)):
        q = {k: v for k, v in p.items() if k not in drop}
        check(bwd(q, s, M, d, rows, **case), q, s, M, rows, **{k: v for k, v in case.items() if k != "skip"})


def test_gradient_against_differences():
    # L = <x, cx> + <r', cr> in float64 along a direction of every input
    M, d, rows = 40, 144, 9
    p = inputs(M, d, rows, seed=5)
    s = saved(p, M, d, rows)
    got = bwd(p, s, M, d, rows)
    cx, cr = s["dx"].to(F64), s["drn"].to(F64)
    base = {k: p[k].to(F64) for k in ("r", "y", "w_post", "gate", "alpha", "w_pre")}

    def loss(q):
        rn, _, x, _ = R.norms_fwd(q["r"], q["y"], q["w_post"], q["gate"], rows, q["alpha"], q["w_pre"], EPS)
        return float((x * cx).sum() + (rn * cr).sum())

    name = {"r": "dr", "y": "dy", "w_post": "dw_post", "gate": "dgate", "alpha": "dalpha", "w_pre": "dw_pre"}
    for i, k in enumerate(base):
        v = torch.randn(base[k].shape, generator=gen(50 + i), device="cuda", dtype=F64)
        h = 1e-5
        num = (loss({**base, k: base[k] + h * v}) - loss({**base, k: base[k] - h * v})) / (2 * h)
        terms = got[name[k]].to(F64) * v
        # BF16 r' in the backward (2^-8 an element) and BF16 gradients: independent roundings
        tol = 2.0 ** -7 * 6 * float(terms.square().sum().sqrt()) + 2.0 ** -8 * abs(num)
        assert abs(float(terms.sum()) - num) <= tol, k


def test_gradient_in_place_and_repeatable():
    M, d, rows = 700, 768, 700
    p = inputs(M, d, rows)
    s = saved(p, M, d, rows)
    a, b = bwd(p, s, M, d, rows), bwd(p, s, M, d, rows)
    assert all(torch.equal(a[k], b[k]) for k in a)  # fixed order of the sums
    dr, dy = s["drn"].clone(), s["dx"].clone()
    ws = torch.empty(A.fp8mlp_norm_gate_bwd_workspace_size(M, d, rows), dtype=U8, device="cuda")
    A.fp8mlp_norm_gate_bwd(M, d, p["r"], p["y"], p["w_post"], p["gate"], rows, p["alpha"], s["rpost"], s["rn"], p["w_pre"],
                           s["rpre"], dy, dr, dr, dy, None, None, None, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(dr, a["dr"]) and torch.equal(dy, a["dy"])


def test_empty_batch_zeroes_the_gains():
    d = 64
    o = [torch.ones(d, device="cuda"), torch.ones(d, device="cuda"), torch.ones(1, device="cuda")]
    A.fp8mlp_norm_gate_bwd(0, d, None, None, None, None, 1, None, None, None, None, None, None, None, None, None, o[0], None,
                           o[2], o[1], None)
    torch.cuda.synchronize()
    assert not any(t.any() for t in o)


def test_captured_replayed_and_on_another_stream():
    M, d, rows = 333, 768, 50
    p = inputs(M, d, rows)
    s = saved(p, M, d, rows)
    want_f, want_b = fwd(p, M, d, rows, quant=True), bwd(p, s, M, d, rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bwd(p, s, M, d, rows, stream=side)
    assert all(torch.equal(got[k], want_b[k]) for k in got)
    outs = [{k: torch.empty_like(v) for k, v in {**want_f, **want_b}.items()} for _ in range(2)]
    ws = [torch.empty(A.fp8mlp_norm_gate_bwd_workspace_size(M, d, rows), dtype=U8, device="cuda") for _ in range(2)]
    graphs = []
    for o, w in zip(outs, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            A.fp8mlp_norm_gate_fwd(M, d, p["r"], p["y"], p["w_post"], p["gate"], rows, p["alpha"], p["w_pre"], EPS,
                                   o["r_next"], o["rstd_post"], o["x"], o["rstd_pre"], o["xq"], o["xs"])
            A.fp8mlp_norm_gate_bwd(M, d, p["r"], p["y"], p["w_post"], p["gate"], rows, p["alpha"], o["rstd_post"],
                                   o["r_next"], p["w_pre"], o["rstd_pre"], s["dx"], s["drn"], o["dr"], o["dy"],
                                   o["dw_post"], o["dgate"], o["dalpha"], o["dw_pre"], w)
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(o[k], v) for k, v in {**want_f, **want_b}.items())


def test_very_many_gate_rows():
    # 2.2 million gate rows of 33: each is shared by several workers
    M, d, rows = 33 * 2_200_000 + 5, 16, 33
    y = torch.randn(M, d, generator=gen(1), device="cuda").to(BF)
    g = torch.randn(R.cdiv(M, rows), d, generator=gen(2), device="cuda").to(BF)
    dr_next = torch.randn(M, d, generator=gen(3), device="cuda").to(BF)
    rpost = torch.rsqrt(y.float().square().mean(1) + EPS)
    dr, dy, dgate = torch.empty_like(y), torch.empty_like(y), torch.full(g.shape, float("nan"), device="cuda")
    ws = torch.empty(A.fp8mlp_norm_gate_bwd_workspace_size(M, d, rows), dtype=U8, device="cuda")
    A.fp8mlp_norm_gate_bwd(M, d, None, y, None, g, rows, None, rpost, None, None, None, None, dr_next, dr, dy, None, dgate,
                           None, None, ws)
    torch.cuda.synchronize()
    t = dr_next[:-5].float() * (y[:-5].float() * rpost[:-5, None])
    want, mag = t.view(-1, rows, d).sum(1), t.view(-1, rows, d).abs().sum(1)
    assert bool(((dgate[:-1] - want).abs() <= ROW * mag).all()) and bool(torch.isfinite(dgate).all())


def test_offsets_beyond_32_bits():
    M, d = 2 ** 31 // 768 + 700, 768
    p = dict(r=torch.empty(M, d, dtype=BF, device="cuda").fill_(0.5), y=torch.empty(M, d, dtype=BF, device="cuda").fill_(0.25))
    p["r"][-50:], p["y"][-50:] = randn(1, 50, d), randn(2, 50, d)
    t = {k: torch.empty(M, d, dtype=BF, device="cuda") for k in ("rn", "x")}
    s1, s2 = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    A.fp8mlp_norm_gate_fwd(M, d, p["r"], p["y"], None, None, M, None, None, EPS, t["rn"], s1, t["x"], s2)
    torch.cuda.synchronize()
    sub = {k: v[-50:].contiguous() for k, v in p.items()}
    want = fwd(sub, 50, d, 50)
    assert torch.equal(t["x"][-50:], want["x"]) and torch.equal(t["rn"][-50:], want["r_next"])
    dr, dy = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    ws = torch.empty(A.fp8mlp_norm_gate_bwd_workspace_size(M, d, M), dtype=U8, device="cuda")
    A.fp8mlp_norm_gate_bwd(M, d, None, p["y"], None, None, M, None, s1, t["rn"], None, s2, t["x"], None, dr, dy, None, None,
                           None, None, ws)
    torch.cuda.synchronize()
    s = dict(rn=want["r_next"], rpost=want["rstd_post"], rpre=want["rstd_pre"], dx=want["x"], drn=None)
    got = bwd(sub, s, 50, d, 50, drn=False)
    assert torch.equal(dr[-50:], got["dr"]) and torch.equal(dy[-50:], got["dy"])


@pytest.mark.parametrize("M,d,rows", [
    # parts by row: a worker's rows are of different gate rows; the last gate row and the last run are short
    (20011, 16, 100), (9001, 32, 60), (5003, 64, 33), (2500, 128, 30), (30011, 16, 128), (65539, 32, 8), (19000, 16, 2),
    (4737, 128, 32), (9473, 64, 64),
    # fewer gate rows than workers, dealt whole; narrow gate rows of more than 32 rows, dealt whole
    (20001, 768, 30), (2500, 768, 4), (1301, 256, 1), (2601, 208, 2), (1200 * 33 + 7, 256, 32), (5000 * 50 + 11, 128, 50),
    (9500 * 60 + 1, 16, 60), (1184, 768, 2), (1183, 768, 2), (18944, 16, 2), (2367, 256, 2), (9472, 64, 2), (16, 768, 2), (8, 768, 2)])
def test_gradient_of_short_gate_rows(M, d, rows):
    p = inputs(M, d, rows, seed=M + d)
    s = saved(p, M, d, rows)
    check(bwd(p, s, M, d, rows), p, s, M, rows)
    skip = bwd(p, s, M, d, rows, skip=("dw_post", "dalpha", "dw_pre"))
    assert torch.equal(skip["dgate"], bwd(p, s, M, d, rows)["dgate"])
