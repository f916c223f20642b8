"""Plain definitions of the block-scaled FP8 product, the gated norms and the
AdamW step, for the tests: elementary torch operations in float64 (in float32,
operation by operation, where the definition fixes the rounding)."""
import torch

E4M3_MAX = 448.0
SCALE_MAX = 2.0 ** 120
F64 = torch.float64


def cdiv(a, b):
    return -(-a // b)


def block_scale(amax):
    """(s, stored 1/s) of blocks with largest magnitude ``amax`` (fp32)."""
    s = torch.full_like(amax, E4M3_MAX).div(amax).clamp(max=SCALE_MAX)
    s = torch.where(amax > 0, s, torch.ones_like(s))
    inv = torch.ones_like(s).div(s)
    bad = ~torch.isfinite(amax)
    return torch.where(bad, torch.ones_like(s), s), torch.where(bad, torch.full_like(s, float("nan")), inv)


def _amax(x, dim):
    """Largest magnitude; NaN if there is one."""
    return x.abs().amax(dim=dim)


def to_codes(x):
    """e4m3 code bytes of fp32 values: nearest, saturating, NaN kept (codes of
    infinities do not matter: their block's scale is NaN)."""
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def quant_rows(x):
    """fp32 [M, K] -> codes [M, K], stored scales [ceil(K/128), M]."""
    M, K = x.shape
    kb = cdiv(K, 128)
    blk = torch.zeros(M, kb * 128, device=x.device)
    blk[:, :K] = x
    blk = blk.view(M, kb, 128)
    s, inv = block_scale(_amax(blk, 2))
    return to_codes((blk * s[:, :, None]).view(M, kb * 128)[:, :K]).contiguous(), inv.t().contiguous()


def quant_weight(W):
    """fp32 [N, K] -> codes [N, K], stored scales [ceil(K/128), ceil(N/128)]."""
    N, K = W.shape
    nb, kb = cdiv(N, 128), cdiv(K, 128)
    pad = torch.zeros(nb * 128, kb * 128, device=W.device)
    pad[:N, :K] = W
    blk = pad.view(nb, 128, kb, 128)
    s, inv = block_scale(_amax(blk, (1, 3)))
    q = (blk * s[:, None, :, None]).reshape(nb * 128, kb * 128)[:N, :K]
    return to_codes(q).contiguous(), inv.t().contiguous()


def row_values(q, s):
    return q.to(F64) * s.to(F64).t().repeat_interleave(128, dim=1)[:, :q.shape[1]]


def weight_values(q, s):
    return q.to(F64) * s.to(F64).t().repeat_interleave(128, dim=0)[:q.shape[0]].repeat_interleave(128, dim=1)[:, :q.shape[1]]


def product(xq, xs, Wq, ws):
    """(exact product, product of magnitudes) in float64."""
    a, b = row_values(xq, xs), weight_values(Wq, ws)
    return a @ b.t(), a.abs() @ b.abs().t()


# ---- norms ----------------------------------------------------------------

def gate_rows(gate, rows, M):
    return gate[torch.arange(M, device=gate.device) // rows]


def norms_fwd(r, y, w_post, gate, rows, alpha, w_pre, eps):
    """float64; y, w_post, gate, alpha, w_pre may be None."""
    M = r.shape[0]
    rpost = None
    rn = r
    if y is not None:
        rpost = 1 / torch.sqrt((y * y).mean(1) + eps)
        t = y * rpost[:, None]
        if w_post is not None:
            t = t * w_post
        if gate is not None:
            t = t * gate_rows(gate, rows, M)
        rn = (1.0 if alpha is None else alpha) * r + t
    rpre = 1 / torch.sqrt((rn * rn).mean(1) + eps)
    x = rn * rpre[:, None]
    return rn, rpost, x if w_pre is None else x * w_pre, rpre


def norms_bwd(r, y, w_post, gate, rows, alpha, rpost, rn, w_pre, rpre, dx, drn):
    """Gradients and, under the same names, the sums of magnitudes that bound
    their rounding errors."""
    M, d = r.shape
    one = torch.ones(d, dtype=F64, device=r.device)
    wpre = one if w_pre is None else w_pre
    wpost = one if w_post is None else w_post
    D = torch.zeros_like(r) if drn is None else drn
    mD = D.abs()
    out, mag = {}, {}
    if dx is not None:
        a = rpre[:, None]
        xh, dxw = rn * a, dx * wpre
        D = D + a * (dxw - xh * (dxw * xh).mean(1, keepdim=True))
        mD = mD + a * (dxw.abs() + xh.abs() * (dxw * xh).abs().mean(1, keepdim=True))
        out["dw_pre"], mag["dw_pre"] = (dx * xh).sum(0), (dx * xh).abs().sum(0)
    al = 1.0 if alpha is None else alpha
    out["dr"], mag["dr"] = al * D, abs(al) * mD
    if y is not None:
        g = one.expand(M, d) if gate is None else gate_rows(gate, rows, M)
        b = rpost[:, None]
        n = y * b
        gw = g * wpost
        dn = D * gw
        out["dy"] = b * (dn - n * (dn * n).mean(1, keepdim=True))
        mag["dy"] = b * (mD * gw.abs() + n.abs() * (mD * (gw * n).abs()).mean(1, keepdim=True))
        out["dw_post"], mag["dw_post"] = (D * g * n).sum(0), (mD * (g * n).abs()).sum(0)
        G = cdiv(M, rows)
        idx = torch.arange(M, device=r.device) // rows
        for k, t in (("out", D * n * wpost), ("mag", mD * (n * wpost).abs())):
            z = torch.zeros(G, d, dtype=F64, device=r.device)
            (out if k == "out" else mag)["dgate"] = z.index_add_(0, idx, t)
        out["dalpha"], mag["dalpha"] = (D * r).sum().view(1), (mD * r.abs()).sum().view(1)
    return out, mag


# ---- AdamW ------------------------------------------------------------------

def f32(v):
    return torch.tensor(v, dtype=torch.float32).item()


def mix32(h):
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def random_bits(n, tensor, step, seed, first=0, device="cpu"):
    key = mix32(torch.tensor((tensor * 0x9E3779B9 + step * 0x7F4A7C15 + seed) & 0xFFFFFFFF, device=device))
    idx = torch.arange(first, first + n, device=device) & 0xFFFFFFFF
    return mix32((mix32(idx ^ key) + key) & 0xFFFFFFFF)


def blocks(x):
    nb = cdiv(x.numel(), 128)
    p = torch.zeros(nb * 128, dtype=x.dtype, device=x.device)
    p[:x.numel()] = x
    return p.view(nb, 128)


def state_values(q, s):
    """fp32 values of 8-bit states."""
    return (blocks(q.float()) * s[:, None]).view(-1)[:q.numel()]


def quant_state(x, u, positive):
    """fp32 [n] -> (codes as values, stored scales), rounded stochastically with u in [0, 1)."""
    b, n = blocks(x), x.numel()
    s, inv = block_scale(b.abs().amax(1))
    a = (b * s[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    q = torch.ldexp(torch.ones_like(a), (torch.frexp(a.abs())[1] - 1).clamp(min=-6) - 3)
    c = torch.sign(a) * (torch.floor(a.abs() / q + blocks(u)) * q).clamp(max=E4M3_MAX)
    if positive:
        c = torch.where((b > 0) & (c == 0), torch.full_like(c, 2.0 ** -9), c)
    return c.view(-1)[:n], inv


def bf16_stochastic(p, bits16):
    w = (((p.view(torch.int32).long() & 0xFFFFFFFF) + bits16) >> 16) << 16
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).view(torch.float32)
    return torch.where(torch.isfinite(p), w, p)


def adamw(p, g, m, v, t, lr, wd, b1, b2, eps, coef=1.0, lr_mult=1.0):
    """One step in fp32, each operation rounded: (p', m', v').  Scalars are
    rounded to fp32 as the call takes them."""
    b1, b2, eps = f32(b1), f32(b2), f32(eps)
    lr = f32(f32(lr) * f32(lr_mult))
    ge = g * f32(coef)
    m = m * b1 + ge * f32(1.0 - b1)
    v = v * b2 + (ge * ge) * f32(1.0 - b2)
    size = f32(lr / (1.0 - b1 ** t))
    inv = f32(1.0 / (1.0 - b2 ** t) ** 0.5)
    p = (p - p * f32(lr * f32(wd))) - (m / (v.sqrt() * inv + eps)) * size
    return p, m, v


def adamw64(p, g, m, v, t, lr, wd, b1, b2, eps):
    """The definition in float64."""
    p, g, m, v = (x.to(F64) for x in (p, g, m, v))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    return p - lr * wd * p - lr / (1 - b1 ** t) * m / (v.sqrt() / (1 - b2 ** t) ** 0.5 + eps), m, v
