"""Plain 64-bit forms (torch on the CPU) of the norms around a branch and of the 4-bit
groups, for the tests, with the magnitudes that bound their rounding."""
import numpy as np
import torch

ULP = 2.0 ** -24  # half a step of fp32, relative


def act(gate, how):
    """The gate's factor, its slope and the size of the slope's terms."""
    if gate is None:
        return torch.ones(()).double(), None, None
    if how is None:
        return gate, torch.ones_like(gate), torch.ones_like(gate)
    p, m = torch.sigmoid(gate), torch.sigmoid(-gate)
    if how == "sigmoid":
        return p, p * m, p * m
    return gate * p, p + gate * p * m, p + (gate * p * m).abs()


def branch(f, nw, eps, gate=None, how=None, alpha=1.0):
    """alpha * a(gate) * f / sqrt(mean f^2 + eps) * nw in float64."""
    r = torch.rsqrt(f.square().mean(1, keepdim=True) + eps)
    return alpha * act(gate, how)[0] * f * r * nw


def site_post_norm(x, f, nw, post, comb, eps, gate=None, how=None, alpha=1.0):
    """The result and the size of its terms."""
    h = branch(f, nw, eps, gate, how, alpha)
    out = post.unsqueeze(2) * h.unsqueeze(1) + comb.transpose(1, 2) @ x
    size = post.abs().unsqueeze(2) * h.abs().unsqueeze(1) + comb.abs().transpose(1, 2) @ x.abs()
    return out, size


def norm_bwd(dz, dz_size, y, nw, eps):
    """dy, dnw of the norm, and bounds of their terms' sizes: what rounds with the row
    (a sum of H terms) and what rounds alone.  dz_size bounds the terms of dz."""
    H = y.shape[1]
    r = torch.rsqrt(y.square().mean(1, keepdim=True) + eps)
    dn = dz * nw
    n = y * r
    dy = r * (dn - n * (dn * n).mean(1, keepdim=True))
    alone = r * dz_size * nw.abs()
    row = y.abs() * r ** 3 / H * (dz_size * nw.abs() * y.abs()).sum(1, keepdim=True)
    return dy, (dz * n).sum(0), alone, row, (dz_size * n.abs()).sum(0)


# ------------------------------------------------------------------ 4-bit groups
def byte_of(col):
    """Byte in a row of codes, and the half of it (0 low, 1 high), of each column."""
    col = np.asarray(col)
    return col // 32 * 16 + col % 16, col % 32 // 16


def pack(c):
    """Codes [N, K] -> bytes [N, K/2]."""
    c = np.asarray(c, np.uint8)
    N, K = c.shape
    out = np.zeros((N, K // 2), np.uint8)
    at, half = byte_of(np.arange(K))
    for k in range(K):
        out[:, at[k]] |= c[:, k] << np.uint8(4 * half[k])
    return out


def unpack(codes, K):
    at, half = byte_of(np.arange(K))
    return (np.asarray(codes)[:, at] >> (4 * half).astype(np.uint8)) & 15


def bf16(v):
    """fp32 values rounded to the nearest bf16, ties to even."""
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).bfloat16().float().numpy()


def encode(w, group, zeros):
    """codes [N, K], scales [N, groups] (fp32 values of bf16), zeros [N, groups]."""
    w = np.asarray(w, np.float32)
    N, K = w.shape
    G = -(-K // group)
    full = np.zeros((N, G * group), np.float32)
    full[:, :K] = w
    b = full.reshape(N, G, group)
    fin = np.where(np.isfinite(b), b, np.float32(0))
    lo, hi = np.minimum(fin.min(2), 0), np.maximum(fin.max(2), 0)
    f = np.float32
    d = bf16(hi / f(15) - lo / f(15)) if zeros else bf16(np.maximum(hi, -lo) / f(7))
    d = np.maximum(d, f(2.0 ** -126))
    z = np.minimum(np.rint(-lo / d), f(15)) if zeros else np.full_like(d, 8)
    with np.errstate(over="ignore", invalid="ignore"):
        c = np.clip(np.rint(b / d[:, :, None]) + z[:, :, None], 0 if zeros else 1, 15)
    c = np.where(np.isnan(b), z[:, :, None], c).astype(np.uint8)
    return c.reshape(N, -1)[:, :K], d, z.astype(np.uint8)


def decode(c, scales, zeros, group):
    """float64 [N, K] of codes [N, K]."""
    g = np.arange(c.shape[1]) // group
    z = 8.0 if zeros is None else np.asarray(zeros, np.float64)[:, g]
    return (np.asarray(c, np.float64) - z) * np.asarray(scales, np.float64)[:, g]
