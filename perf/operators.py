"""Cases that measure three operators of a training step of an MLP stack:

- the FP8 matrix product with a scale for each block of 128 (``linear``: a
  layer's forward from BF16 activations; ``dx``: the input gradient from the
  transposed weight cache; ``mlp``: up-projection, relu^2 and down-projection),
- the norms after one block and before the next, fused with the gate and the
  residual scale (``norms_fwd``, ``norms_bwd``),
- the AdamW step over many tensors with its gradient norm (``adamw``).

``own`` selects between elementary torch operations (False) and the package's
kernels (True); both take what ``prepare`` returns.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_MAX = 2.0 ** 120
EPS = 1e-6  # of the norms
BETA1, BETA2, ADAM_EPS = 0.9, 0.95, 1e-8
MAX_NORM = 1.0


def cdiv(a, b):
    return -(-a // b)


def _scale(amax):
    """fp32 factor that maps a block's largest magnitude onto 448 (one division, rounded once)."""
    s = torch.full_like(amax, E4M3_MAX).div(amax).clamp(max=SCALE_MAX)
    return torch.where(amax > 0, s, torch.ones_like(s))


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token through a QKV projection: launch latency and the weight's bytes
        {"name": "linear_token", "op": "linear", "M": 1, "K": 768, "N": 2304},
        # the QKV projection of one training step of 16384 tokens
        {"name": "linear_qkv16k", "op": "linear", "M": 16384, "K": 768, "N": 2304},
        # input gradient of a layer with ragged rows and columns
        {"name": "dx_ragged", "op": "dx", "M": 5003, "K": 1040, "N": 2320},
        # a whole MLP forward, hidden layer of four times the width
        {"name": "mlp_8k", "op": "mlp", "M": 8192, "d": 1024, "h": 4096},
        # one token between two blocks
        {"name": "norms_fwd_token", "op": "norms_fwd", "M": 1, "d": 768, "rows": 1, "quant": True},
        # a training step between two blocks, one learned gate vector
        {"name": "norms_fwd_16k", "op": "norms_fwd", "M": 16384, "d": 768, "rows": 16384, "quant": True},
        # its gradient
        {"name": "norms_bwd_16k", "op": "norms_bwd", "M": 16384, "d": 768, "rows": 16384},
        # a wider stream of uneven length, one gate vector per sequence of 1000 tokens
        {"name": "norms_bwd_ragged", "op": "norms_bwd", "M": 7777, "d": 2064, "rows": 1000},
        # many small and odd tensors (norm gains, gates, biases): latency
        {"name": "adamw32_small", "op": "adamw", "bits": 32, "master": True, "matrices": 0, "size": 0, "vectors": 60,
         "odd": 1537},
        # nine layers of up- and down-projections, states in 32 bits
        {"name": "adamw32_stack9", "op": "adamw", "bits": 32, "master": True, "matrices": 18, "size": 2359296,
         "vectors": 18, "odd": 768},
        # the same with states in 8 bits
        {"name": "adamw8_stack9", "op": "adamw", "bits": 8, "master": True, "matrices": 18, "size": 2359296,
         "vectors": 18, "odd": 768},
        # a vocabulary head in BF16 alone (no 32-bit weights), states in 8 bits
        {"name": "adamw8_head", "op": "adamw", "bits": 8, "master": False, "matrices": 1, "size": 50304 * 768,
         "vectors": 3, "odd": 50303},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, min(int(hi) // step * step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "dx", "mlp", "norms_fwd", "norms_bwd", "adamw", "adamw"])
    if op in ("linear", "dx"):
        return {"op": op, "M": _log(rng, 1, 16384), "K": _log(rng, 16, 2048, 16), "N": _log(rng, 16, 2048, 16)}
    if op == "mlp":
        d = _log(rng, 16, 1024, 16)
        return {"op": op, "M": _log(rng, 1, 8192), "d": d, "h": min(4096, 16 * rng.randint(d // 16, 4 * d // 16))}
    if op.startswith("norms"):
        M, d = _log(rng, 1, 16384), _log(rng, 16, 4096, 16)
        M = max(1, min(M, 16000000 // d))
        rows = rng.choice([1, _log(rng, 1, M), M])
        c = {"op": op, "M": M, "d": d, "rows": rows}
        return dict(c, quant=rng.random() < 0.5) if op == "norms_fwd" else c
    return {"op": op, "bits": rng.choice([8, 32]), "master": rng.random() < 0.7, "matrices": rng.randint(1, 12),
            "size": _log(rng, 256, 3000000), "vectors": rng.randint(0, 40), "odd": _log(rng, 1, 5000)}


def _sizes(case):
    return [case["size"]] * case["matrices"] + [case["odd"]] * case["vectors"]


def work(case):
    op = case["op"]
    if op in ("linear", "dx"):
        M, K, N = (case[k] for k in ("M", "K", "N"))
        if op == "dx":
            K, N = N, K
        # x in, its codes and scales out, the weight's codes, y out
        return {"bytes": M * K * 3 + 4 * M * cdiv(K, 128) + N * K + M * N * 2, "flops": 2 * M * N * K}
    if op == "mlp":
        M, d, h = case["M"], case["d"], case["h"]
        return {"bytes": M * d * 3 + 4 * M * cdiv(d, 128) + 2 * h * d + M * h * 3 + 4 * M * cdiv(h, 128) + M * d * 2,
                "flops": 4 * M * d * h}
    if op == "norms_fwd":
        M, d = case["M"], case["d"]
        q = M * d + 4 * M * cdiv(d, 128) if case["quant"] else 0
        return {"bytes": 8 * M * d + 8 * M + 2 * cdiv(M, case["rows"]) * d + q, "flops": 12 * M * d}
    if op == "norms_bwd":
        M, d = case["M"], case["d"]
        return {"bytes": 14 * M * d + 8 * M + 6 * cdiv(M, case["rows"]) * d, "flops": 30 * M * d}
    n = sum(_sizes(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / 128
    # the gradient is read for its norm, which the step needs, and by the step
    return {"bytes": n * (8 + (8 if case["master"] else 0) + (2 if case["master"] else 4) + state), "flops": 20 * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _weight_cache(W):
    """e4m3 codes of W [N, K] and the inverse scales [K/128, N/128] of its 128 x 128 blocks."""
    N, K = W.shape
    nb, kb = cdiv(N, 128), cdiv(K, 128)
    pad = torch.zeros(nb * 128, kb * 128, device=W.device)
    pad[:N, :K] = W.float()
    blk = pad.view(nb, 128, kb, 128)
    amax = blk.abs().amax(dim=(1, 3))
    s = _scale(amax)
    q = (blk * s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).reshape(nb * 128, kb * 128)[:N, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), (1.0 / s).t().contiguous()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    bf, u8, f32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32

    def randn(*shape, scale=1.0, dtype=bf):
        return (torch.randn(*shape, generator=g, device=dev, dtype=f32) * scale).to(dtype)

    def act(M, K, scale=1.0):  # activations: a few channels are much larger than the rest
        t = torch.randn(M, K, generator=g, device=dev)
        big = torch.rand(K, generator=g, device=dev) < 0.01
        return (t * torch.where(big, 20.0, 1.0) * scale).to(bf)

    op = case["op"]
    s = {"case": case}
    if op in ("linear", "dx"):
        M, K, N = case["M"], case["K"], case["N"]
        W = randn(N, K, scale=K ** -0.5)
        if op == "dx":  # the product runs over the layer's N with the transposed cache
            W, K, N = W.t().contiguous(), N, K
        x = act(M, K, 1.0 if op == "linear" else 1e-4)
        Wq, ws = _weight_cache(W)
        s.update(x=x, Wq=Wq, ws=ws, xq=torch.empty(M, K, dtype=u8, device=dev),
                 xs=torch.empty(cdiv(K, 128), M, device=dev), y=torch.empty(M, N, dtype=bf, device=dev))
    elif op == "mlp":
        M, d, h = case["M"], case["d"], case["h"]
        W1q, w1s = _weight_cache(randn(h, d, scale=d ** -0.5))
        W2q, w2s = _weight_cache(randn(d, h, scale=h ** -0.5))
        s.update(x=act(M, d), W1q=W1q, w1s=w1s, W2q=W2q, w2s=w2s, xq=torch.empty(M, d, dtype=u8, device=dev),
                 xs=torch.empty(cdiv(d, 128), M, device=dev), post=torch.empty(M, h, dtype=bf, device=dev),
                 postq=torch.empty(M, h, dtype=u8, device=dev), posts=torch.empty(cdiv(h, 128), M, device=dev),
                 out=torch.empty(M, d, dtype=bf, device=dev))
    elif op.startswith("norms"):
        M, d, rows = case["M"], case["d"], case["rows"]
        G = cdiv(M, rows)
        s.update(r=act(M, d, 3.0), y=randn(M, d, scale=0.3), wpost=(1 + randn(d, scale=0.1, dtype=f32)).to(bf),
                 wpre=(1 + randn(d, scale=0.1, dtype=f32)).to(bf), gate=(0.5 + randn(G, d, scale=0.2, dtype=f32)).to(bf),
                 alpha=0.9 + randn(1, scale=0.05, dtype=f32), rpost=torch.empty(M, device=dev),
                 rpre=torch.empty(M, device=dev))
        if op == "norms_fwd":
            s.update(rnext=torch.empty(M, d, dtype=bf, device=dev), x=torch.empty(M, d, dtype=bf, device=dev))
            if case["quant"]:
                s.update(xq=torch.empty(M, d, dtype=u8, device=dev), xs=torch.empty(cdiv(d, 128), M, device=dev))
        else:
            # what the forward left: the next residual stream and both norms' statistics
            rn, _, rpost, rpre = _norms(s["r"].float(), s["y"].float(), s["wpost"].float(), s["gate"].float(), rows,
                                        s["alpha"], s["wpre"].float())
            s.update(rnext=rn.to(bf), rpost=rpost, rpre=rpre, dx=randn(M, d, scale=1e-3), drn=randn(M, d, scale=1e-3),
                     dr=torch.empty(M, d, dtype=bf, device=dev), dy=torch.empty(M, d, dtype=bf, device=dev),
                     dwpost=torch.empty(d, device=dev), dwpre=torch.empty(d, device=dev),
                     dgate=torch.empty(G, d, device=dev), dalpha=torch.empty(1, device=dev))
            if own:
                from fp8_relu_mlp_b200 import _abi as A
                s["workspace"] = torch.empty(max(16, A.fp8mlp_norm_gate_bwd_workspace_size(M, d, rows)),
                                             dtype=torch.uint8, device=dev)
    else:
        sizes = _sizes(case)
        off, total = [], 0
        for n in sizes:
            off.append(total)
            total += cdiv(n, 128) * 128
        nb = total // 128
        ok = torch.zeros(total, dtype=torch.bool, device=dev)  # False in the padding between tensors
        tid = torch.zeros(total, dtype=torch.int64, device=dev)  # tensor of each element, and its index there
        idx = torch.arange(total, device=dev)
        for i, (o, n) in enumerate(zip(off, sizes)):
            ok[o:o + n] = True
            tid[o:o + cdiv(n, 128) * 128] = i
            idx[o:o + cdiv(n, 128) * 128] -= o
        z = torch.zeros((), device=dev)
        # gradients of very different sizes within a tensor; moments as after some steps
        mag = torch.exp(1.5 * torch.randn(total, generator=g, device=dev)) * 1e-4
        grad = torch.where(ok, torch.randn(total, generator=g, device=dev) * mag, z)
        m = torch.where(ok, 0.2 * torch.randn(total, generator=g, device=dev) * mag, z)
        v = torch.where(ok, mag * mag * (0.5 + torch.rand(total, generator=g, device=dev)), z)
        p = torch.where(ok, torch.randn(total, generator=g, device=dev) * 0.02, z)
        s.update(sizes=sizes, off=off, grad=grad, p16=p.to(bf), p=p if case["master"] else None, ok=ok, tid=tid, idx=idx,
                 step=torch.full((1,), 10, dtype=torch.int32, device=dev), lr=1e-3, wd=0.1, seed=int(seed) & 0x7FFFFFFF,
                 norm=torch.empty(2, device=dev))
        if case["bits"] == 32:
            s.update(m=m, v=v)
        else:
            mq, ms = _quant_state(m, nb, None, False)
            vq, vs = _quant_state(v.sqrt(), nb, None, True)
            s.update(m=mq, v=vq, ms=ms, vs=vs)
        if own:
            from fp8_relu_mlp_b200.optim import AdamW
            opt = AdamW(state_bits=case["bits"], lr=s["lr"], betas=(BETA1, BETA2), eps=ADAM_EPS, seed=s["seed"],
                        max_norm=MAX_NORM, step_count=10)
            for o, n in zip(off, sizes):
                b = cdiv(n, 128)
                st = {"m": s["m"][o:o + n], "v": s["v"][o:o + n]}
                if case["bits"] == 8:
                    st.update(m_scale=s["ms"][o // 128:o // 128 + b], v_scale=s["vs"][o // 128:o // 128 + b])
                opt.add(grad=grad[o:o + n], master=p[o:o + n] if case["master"] else None, weight=s["p16"][o:o + n],
                        weight_decay=s["wd"], state=st)
            s["opt"] = opt
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _quant_rows(x):
    """fp32 [M, K] -> e4m3 codes and inverse scales [K/128, M] of groups of 128 along K."""
    M, K = x.shape
    kb = cdiv(K, 128)
    blk = torch.nn.functional.pad(x, (0, kb * 128 - K)).view(M, kb, 128)
    amax = blk.abs().amax(dim=2)
    s = _scale(amax)
    q = (blk * s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(M, kb * 128)[:, :K]
    return q.to(torch.float8_e4m3fn), (1.0 / s).t().contiguous()


def _values(q, s_rows):
    """What row-quantised codes stand for, fp32."""
    return q.float() * s_rows.t().repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _weight_values(q, s):
    N, K = q.shape
    return q.float() * s.t().repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)[:, :K]


def _norms(r, y, wpost, gate, rows, alpha, wpre):
    gate = gate.repeat_interleave(rows, dim=0)[:r.shape[0]]
    rpost = torch.rsqrt((y * y).mean(dim=1) + EPS)
    rn = alpha * r + gate * (y * rpost[:, None] * wpost)
    rpre = torch.rsqrt((rn * rn).mean(dim=1) + EPS)
    return rn, rn * rpre[:, None] * wpre, rpost, rpre


def _group_sum(t, rows):
    """Sum of the rows of each group of `rows` rows, the last one shorter."""
    M, d = t.shape
    G = cdiv(M, rows)
    if G == M:
        return t
    out = t[:(M // rows) * rows].view(M // rows, rows, d).sum(dim=1)
    return out if M % rows == 0 else torch.cat([out, t[(M // rows) * rows:].sum(dim=0, keepdim=True)])


def _mix(h):
    """The 32-bit finaliser of MurmurHash3, on int64 holding 32-bit values."""
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random_bits(idx, tid, seed, step):
    """32 bits per element: a function of (seed, step, tensor, index)."""
    key = _mix((tid * 0x9E3779B9 + step * 0x7F4A7C15 + seed) & 0xFFFFFFFF)
    return _mix((_mix(idx ^ key) + key) & 0xFFFFFFFF)


def _quant_state(t, nb, u, positive):
    """Blocks of 128 values -> e4m3 codes and inverse scales; `u` in [0, 1) rounds stochastically, None to nearest.
    With `positive` a value above zero never becomes zero."""
    blk = t.view(nb, 128)
    amax = blk.abs().amax(dim=1)
    s = _scale(amax)
    a = (blk * s[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    if u is not None:
        e = (torch.frexp(a.abs())[1] - 1).clamp(min=-6)
        q = torch.ldexp(torch.ones_like(a), e - 3)
        a = torch.sign(a) * (torch.floor(a.abs() / q + u.view(nb, 128)) * q).clamp(max=E4M3_MAX)
    c = a.to(torch.float8_e4m3fn).float()
    if positive:
        c = torch.where((blk > 0) & (c == 0), torch.full_like(c, 2.0 ** -9), c)
    return c.to(torch.float8_e4m3fn).view(-1), 1.0 / s


def _plain_adamw(s):
    case = s["case"]
    g = s["grad"]
    norm = g.double().square().sum().sqrt()
    coef = (MAX_NORM / (norm.float() + 1e-6)).clamp(max=1.0)
    s["norm"].copy_(torch.stack([norm.float(), coef]))
    step = s["step"]
    step += 1
    t = step.double()
    lr = _f32(s["lr"])
    size = (lr / (1 - BETA1_F ** t)).float()
    inv = (1 / torch.sqrt(1 - BETA2_F ** t)).float()
    decay = _f32(lr * _f32(s["wd"]))
    nb = g.numel() // 128
    ge = g * coef
    if case["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].view(nb, 128).float() * s["ms"][:, None]).view(-1)
        u = (s["v"].view(nb, 128).float() * s["vs"][:, None]).view(-1)
        v = u * u
    m = m * BETA1_F + ge * OM_BETA1
    v = v * BETA2_F + (ge * ge) * OM_BETA2
    p = s["p"] if case["master"] else s["p16"].float()
    p = (p - p * decay) - (m / (torch.sqrt(v) * inv + ADAM_EPS_F)) * size
    bits = None
    if case["bits"] == 8 or not case["master"]:
        bits = _random_bits(s["idx"], s["tid"], s["seed"], step.long())
    if case["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        um, uv = (bits & 0xFFFF).float() * 2.0 ** -16, (bits >> 16).float() * 2.0 ** -16
        mq, ms = _quant_state(m, nb, um, False)
        vq, vs = _quant_state(torch.sqrt(v), nb, uv, True)
        s["m"].copy_(mq)
        s["v"].copy_(vq)
        s["ms"].copy_(ms)
        s["vs"].copy_(vs)
    if case["master"]:
        s["p"].copy_(p)
        s["p16"].copy_(p)
    else:  # BF16 alone: rounded stochastically with bits of its own
        low = _mix(bits ^ 0x5BD1E995) & 0xFFFF
        w = ((p.view(torch.int32).long() & 0xFFFFFFFF) + low) >> 16 << 16
        w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).view(torch.float32)
        s["p16"].copy_(torch.where(s["ok"], w, torch.zeros_like(w)))


def _f32(v):
    return torch.tensor(v, dtype=torch.float32).item()


BETA1_F, BETA2_F, ADAM_EPS_F = _f32(BETA1), _f32(BETA2), _f32(ADAM_EPS)
OM_BETA1, OM_BETA2 = _f32(1.0 - BETA1_F), _f32(1.0 - BETA2_F)  # rounded once from 1 - beta


def run(s):
    case = s["case"]
    op = case["op"]
    if op in ("linear", "dx"):
        if own:
            from fp8_relu_mlp_b200 import _abi as A
            M, K = s["x"].shape
            A.fp8mlp_linear_block(M, K, s["Wq"].shape[0], s["x"], s["Wq"], s["ws"], s["xq"], s["xs"], s["y"])
            return {"xq": s["xq"], "xs": s["xs"], "y": s["y"]}
        xq, xs = _quant_rows(s["x"].float())
        y = _values(xq, xs) @ _weight_values(s["Wq"], s["ws"]).t()
        return {"xq": xq, "xs": xs, "y": y.to(torch.bfloat16)}
    if op == "mlp":
        if own:
            from fp8_relu_mlp_b200 import _abi as A
            A.fp8mlp_mlp_fwd_block(case["M"], case["d"], case["h"], s["x"], s["W1q"], s["w1s"], s["W2q"], s["w2s"],
                                   s["xq"], s["xs"], s["post"], s["postq"], s["posts"], s["out"])
            return {"post": s["post"], "postq": s["postq"], "posts": s["posts"], "out": s["out"]}
        xq, xs = _quant_rows(s["x"].float())
        post = (_values(xq, xs) @ _weight_values(s["W1q"], s["w1s"]).t()).clamp(min=0).square()
        postq, posts = _quant_rows(post)
        out = _values(postq, posts) @ _weight_values(s["W2q"], s["w2s"]).t()
        return {"post": post.to(torch.bfloat16), "postq": postq, "posts": posts, "out": out.to(torch.bfloat16)}
    if op == "norms_fwd":
        names = ("rnext", "x", "rpost", "rpre") + (("xq", "xs") if case["quant"] else ())
        if own:
            from fp8_relu_mlp_b200 import _abi as A
            A.fp8mlp_norm_gate_fwd(case["M"], case["d"], s["r"], s["y"], s["wpost"], s["gate"], case["rows"],
                                   s["alpha"], s["wpre"], EPS, s["rnext"], s["rpost"], s["x"], s["rpre"],
                                   s.get("xq"), s.get("xs"))
            return {k: s[k] for k in names}
        rn, x, rpost, rpre = _norms(s["r"].float(), s["y"].float(), s["wpost"].float(), s["gate"].float(),
                                    case["rows"], s["alpha"], s["wpre"].float())
        out = {"rnext": rn.to(torch.bfloat16), "x": x.to(torch.bfloat16), "rpost": rpost, "rpre": rpre}
        if case["quant"]:
            out["xq"], out["xs"] = _quant_rows(x)
        return out
    if op == "norms_bwd":
        if own:
            from fp8_relu_mlp_b200 import _abi as A
            A.fp8mlp_norm_gate_bwd(case["M"], case["d"], s["r"], s["y"], s["wpost"], s["gate"], case["rows"],
                                   s["alpha"], s["rpost"], s["rnext"], s["wpre"], s["rpre"], s["dx"], s["drn"],
                                   s["dr"], s["dy"], s["dwpost"], s["dgate"], s["dalpha"], s["dwpre"], s["workspace"])
            return {k: s[k] for k in ("dr", "dy", "dwpost", "dgate", "dalpha", "dwpre")}
        rows, wpost = case["rows"], s["wpost"].float()
        gate = s["gate"].float().repeat_interleave(rows, dim=0)[:case["M"]]
        xhat = s["rnext"].float() * s["rpre"][:, None]
        dx = s["dx"].float()
        dxw = dx * s["wpre"].float()
        D = s["drn"].float() + s["rpre"][:, None] * (dxw - xhat * (dxw * xhat).mean(dim=1, keepdim=True))
        n = s["y"].float() * s["rpost"][:, None]
        dn = D * gate * wpost
        dy = s["rpost"][:, None] * (dn - n * (dn * n).mean(dim=1, keepdim=True))
        return {"dr": (s["alpha"] * D).to(torch.bfloat16), "dy": dy.to(torch.bfloat16),
                "dwpost": (D * gate * n).double().sum(dim=0).float(),
                "dgate": _group_sum((D * n * wpost).double(), rows).float(),
                "dalpha": (D.double() * s["r"].double()).sum().float().view(1),
                "dwpre": (dx * xhat).double().sum(dim=0).float()}
    if own:
        s["opt"].step()
        s["norm"] = s["opt"].norm
    else:
        _plain_adamw(s)
    names = ["norm", "p16", "m", "v"] + (["p"] if case["master"] else []) + (["ms", "vs"] if case["bits"] == 8 else [])
    return {k: s[k] for k in names}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _e4m3_64(a):
    """Nearest e4m3 value (ties to even), in float64."""
    _, e = torch.frexp(a.abs())
    q = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-6) - 3)
    return (torch.round(a / q) * q).clamp(-E4M3_MAX, E4M3_MAX)


def _codes_64(x):
    """(codes, inverse scales [..., 1]) of float64 x [..., 128].  The scale and the scaled value are 32-bit numbers by
    definition, which decides between two codes where a value is halfway between them."""
    top = x.abs().amax(dim=-1, keepdim=True)
    s = torch.where(top > 0, torch.minimum(E4M3_MAX / top, torch.full_like(top, SCALE_MAX)), torch.ones_like(top))
    s = s.float().double()
    return _e4m3_64((x * s).float().double()), 1 / s


def _rows_64(x):
    M, K = x.shape
    kb = cdiv(K, 128)
    pad = torch.zeros(M, kb * 128, dtype=torch.float64, device=x.device)
    pad[:, :K] = x
    c, inv = _codes_64(pad.view(M, kb, 128))
    val = (c * inv).view(M, kb * 128)[:, :K]
    return c.view(M, kb * 128)[:, :K], inv[:, :, 0].t(), val


def _weight_64(q, s):
    n = torch.arange(q.shape[0], device=q.device) // 128
    k = torch.arange(q.shape[1], device=q.device) // 128
    return q.double() * s.double()[k][:, n].t()


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("linear", "dx"):
        c, inv, val = _rows_64(s["x"].double())
        return {"xq": c, "xs": inv, "y": val @ _weight_64(s["Wq"], s["ws"]).t()}
    if op == "mlp":
        _, _, val = _rows_64(s["x"].double())
        post = torch.relu(val @ _weight_64(s["W1q"], s["w1s"]).t()) ** 2
        c, inv, val = _rows_64(post)
        return {"post": post, "postq": c, "posts": inv, "out": val @ _weight_64(s["W2q"], s["w2s"]).t()}
    if op.startswith("norms"):
        r, y, wpost, gate, wpre = (s[k].double() for k in ("r", "y", "wpost", "gate", "wpre"))
        alpha = s["alpha"].double()
        gate = gate[torch.arange(case["M"], device=r.device) // case["rows"]]
        if op == "norms_fwd":
            rpost = 1 / torch.sqrt(torch.mean(y ** 2, 1) + EPS)
            rn = alpha * r + gate * wpost * y * rpost.unsqueeze(1)
            rpre = 1 / torch.sqrt(torch.mean(rn ** 2, 1) + EPS)
            x = wpre * rn * rpre.unsqueeze(1)
            out = {"rnext": rn, "x": x, "rpost": rpost, "rpre": rpre}
            if case["quant"]:
                out["xq"], out["xs"], _ = _rows_64(x)
            return out
        d = case["d"]
        a, b = s["rpre"].double().unsqueeze(1), s["rpost"].double().unsqueeze(1)
        dx, xh, n = s["dx"].double(), s["rnext"].double() * a, y * b
        D = s["drn"].double() + a * (wpre * dx - xh * ((wpre * dx * xh).sum(1, keepdim=True) / d))
        t = D * gate * wpost
        G = cdiv(case["M"], case["rows"])
        dgate = torch.zeros(G, d, dtype=torch.float64, device=r.device)
        dgate.index_add_(0, torch.arange(case["M"], device=r.device) // case["rows"], D * n * wpost)
        return {"dr": alpha * D, "dy": b * (t - n * ((t * n).sum(1, keepdim=True) / d)), "dwpost": (D * gate * n).sum(0),
                "dgate": dgate, "dalpha": (D * r).sum().view(1), "dwpre": (dx * xh).sum(0)}
    bits8, master = case["bits"] == 8, case["master"]
    g = s["grad"].double()
    norm = torch.sqrt(torch.sum(g * g))
    coef = torch.minimum(MAX_NORM / (norm + 1e-6), torch.ones_like(norm))
    g = g * coef
    if bits8:
        m = s["m"].double().view(-1, 128) * s["ms"].double()[:, None]
        v = (s["v"].double().view(-1, 128) * s["vs"].double()[:, None]) ** 2
        m, v = m.reshape(-1), v.reshape(-1)
    else:
        m, v = s["m"].double(), s["v"].double()
    m = BETA1_F * m + (1 - BETA1_F) * g
    v = BETA2_F * v + (1 - BETA2_F) * g * g
    p = s["p"].double() if master else s["p16"].double()
    t, lr = 11, _f32(s["lr"])
    p = p * (1 - lr * _f32(s["wd"])) - lr * (m / (1 - BETA1_F ** t)) / (torch.sqrt(v / (1 - BETA2_F ** t)) + ADAM_EPS_F)
    out = {"norm": torch.stack([norm, coef]), "p16": p}
    if master:
        out["p"] = p
    if not bits8:
        return dict(out, m=m, v=v)
    r = _random_bits(s["idx"], s["tid"], s["seed"], 11)

    def states(x, u, positive):
        x = x.view(-1, 128)
        top = x.abs().amax(dim=1, keepdim=True)
        sc = torch.where(top > 0, torch.minimum(E4M3_MAX / top, torch.full_like(top, SCALE_MAX)), torch.ones_like(top))
        a = (x * sc).abs()
        q = torch.ldexp(torch.ones_like(a), (torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
        c = (torch.floor(a / q + u.view(-1, 128).double() / 65536) * q).clamp(max=E4M3_MAX)
        if positive:
            c = torch.where((x > 0) & (c == 0), torch.full_like(c, 2.0 ** -9), c)
        return (torch.sign(x) * c).view(-1), (1 / sc).view(-1)

    out["m"], out["ms"] = states(m, r & 0xFFFF, False)
    out["v"], out["vs"] = states(torch.sqrt(v), r >> 16, True)
    return out
