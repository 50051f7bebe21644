"""Plain 64-bit forms (numpy / torch on the CPU) of the 8-bit blocks and of the
site's backward passes, for the tests."""
import numpy as np
import torch

BLOCK = 128

# the finite e4m3 magnitudes in code order: subnormals k * 2^-9, then
# (8 + mantissa) / 8 * 2^(exponent - 7); code 0x7f is NaN
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) / 8 * 2.0 ** ((c >> 3) - 7)
                 for c in range(127)])


def up(n):
    return -(-n // BLOCK) * BLOCK


def e4m3_codes(v):
    """Codes (uint8) of float64 values: nearest magnitude, ties to the even code."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == 0, 0, code).astype(np.uint8)
    code[~np.isfinite(v)] = 0x7f
    return code | (np.signbit(v) << 7).astype(np.uint8)


def scale_exponent(a):
    """Least integer e >= -126 with a <= 448 * 2^e; 0 for a = 0."""
    if a == 0:
        return 0
    e = -126
    f, p = np.frexp(a)
    e = max(e, int(p) - 10)
    while a > 448.0 * 2.0 ** e:
        e += 1
    return e


def encode(x, square=False):
    """x [rows, cols] -> (codes uint8 [rows, P], scale bytes)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    tall = BLOCK if square else 1
    full = np.zeros((-(-rows // tall) * tall, up(cols)))
    full[:rows, :cols] = x
    blocks = full.reshape(full.shape[0] // tall, tall, -1, BLOCK)
    size = np.where(np.isfinite(blocks), np.abs(blocks), 0.0).max((1, 3))
    e = np.array([[scale_exponent(a) for a in r] for r in size]).reshape(size.shape)
    with np.errstate(invalid="ignore"):
        codes = e4m3_codes(blocks * 2.0 ** -e[:, None, :, None].astype(np.float64))
    return codes.reshape(full.shape)[:rows], (e + 127).astype(np.uint8)


def decode(codes, scales, cols, square=False):
    """Values as fp32 holds them: exact, but for code 256 and more at e = 120 (entries
    above 248 * 2^120 round there), which is 2^128 or more and therefore infinite."""
    codes = np.asarray(codes, np.uint8)
    v = np.append(E4M3, np.nan)[codes & 0x7f] * np.where(codes & 0x80, -1.0, 1.0)
    s = 2.0 ** (np.asarray(scales, np.float64) - 127)
    if square:
        s = np.repeat(s, BLOCK, 0)[:codes.shape[0]]
    with np.errstate(over="ignore"):
        return (v * np.repeat(s, BLOCK, 1))[:, :cols].astype(np.float32).astype(np.float64)


def site_pre(x, w, scale, base, iters, eps):
    """The pre chain in torch float64 (differentiable): pre, post, comb, y."""
    T, S, H = x.shape
    flat = x.reshape(T, S * H)
    m = flat @ w.t() * torch.rsqrt(flat.square().mean(1, keepdim=True) + eps)
    z = torch.cat([m[:, :S] * scale[0], m[:, S:2 * S] * scale[1], m[:, 2 * S:] * scale[2]],
                  1) + base
    pre, post = torch.sigmoid(z[:, :S]), 2 * torch.sigmoid(z[:, S:2 * S])
    c = torch.exp(z[:, 2 * S:]).reshape(T, S, S)
    for _ in range(iters):
        c = c / (c.sum(2, keepdim=True) + eps)
        c = c / (c.sum(1, keepdim=True) + eps)
    return pre, post, c, (pre.unsqueeze(2) * x).sum(1)


def site_post(x, f, post, comb):
    return post.unsqueeze(2) * f.unsqueeze(1) + comb.transpose(1, 2) @ x


def pre_grads(x, w, scale, base, iters, eps, dy, dpre, dpost, dcomb, dx_in):
    """dx, dfn_w, dscale, dbase of the pre chain by automatic differentiation in float64."""
    leaves = [t.double().clone().requires_grad_() for t in (x, w, scale, base)]
    outs = site_pre(*leaves, iters, eps)
    seeds = [dpre, dpost, dcomb, dy]
    torch.autograd.backward([o for o, s in zip(outs, seeds) if s is not None],
                            [s.double() for s in seeds if s is not None])
    grads = [t.grad for t in leaves]
    if dx_in is not None:
        grads[0] = grads[0] + dx_in.double()
    return grads
