"""Inputs of site_pre_bwd on which the low bits of its fp32 products are all that is left:
one product of two 24-bit values and the fp32 value nearest to it with the other sign, so
that the sum is the product's own rounding error.  Its exact value is known in 64 bits,
and whatever the call's arithmetic leaves out of the product shows whole.

Of the products of three bf16 planes each the call leaves out p1 p2, p2 p1 and p2 p2: at
most KEPT of the product (planes rounded to nearest: |p1| <= 2^-8 and |p2| <= 2^-17 of a
value in [1, 2))."""
import torch

KEPT = 2.0 ** -24 * (1 + 2.0 ** -9)
# The fp32 sums that lead to the small one: once the leading planes have cancelled what is
# left is at most 2^-6 of the product, and each of at most eight additions is off by at most
# a unit in its last place (2^-23 of it)
SUMS = 8 * 2.0 ** -6 * 2.0 ** -23


def rand24(gen, *shape):
    """fp32 values of both signs in [1, 2), all 24 bits in use; every eighth one of those
    whose planes lose the most when they are cut: 1 + 2^-7 - 2^-23 and its neighbours."""
    k = torch.randint(0, 1 << 23, shape, generator=gen)
    hard = (1 << 16) - 1 - torch.randint(0, 64, shape, generator=gen)
    k = torch.where(torch.randint(0, 8, shape, generator=gen) == 0, hard, k)
    sign = 1.0 - 2.0 * torch.randint(0, 2, shape, generator=gen)
    return ((1 + k.double() * 2.0 ** -23) * sign).float()


def pair(a, b):
    """c = the fp32 value nearest to a b, and a b - c in 64 bits (exact)."""
    ab = a.double() * b.double()
    c = ab.float()
    return c, ab - c.double()


def dots(T, S, H, seed, f8):
    """A pre gate a token and stream whose dot is a b - c (f8: a 1 - c, c = a rounded to 18
    bits, since x is 1 or -1).  dy is one column in which x is zero: dx there is the gate."""
    g = torch.Generator().manual_seed(seed)
    x, w = torch.zeros(T, S, H), torch.zeros((2 + S) * S, S, H)
    want, size = torch.zeros(T, S, dtype=torch.float64), torch.zeros(T, S, dtype=torch.float64)
    for r in range(S):
        at = 2 * int(torch.randint(0, H // 2 - 1, (), generator=g))
        a = rand24(g, 1)
        if f8:
            b = torch.ones(T)
            c = (a.double() * 2.0 ** 17).round().float() * 2.0 ** -17
            w[r, r, at], w[r, r, at + 1] = a, c
            x[:, r, at], x[:, r, at + 1] = 1.0, -1.0
            want[:, r] = (a.double() - c.double()) * b.double()
        else:
            b = rand24(g, T)
            c, want[:, r] = pair(a, b)
            w[r, r, at], w[r, r, at + 1] = a, 1.0
            x[:, r, at], x[:, r, at + 1] = b, -c
        size[:, r] = (a.double() * b.double()).abs()
    dy = torch.zeros(T, H)
    dy[:, H - 1] = 1.0
    return dict(x=x, w=w.reshape((2 + S) * S, S * H), dy=dy, want=want, size=size)


def seeds(u, S):
    """Gradients of the gates that make u [T, R] the call's own u (times 2^-20), exactly, with
    base = 0, iters = 1, eps = 2^40 and dots so small, or a scale, that every gate is 1/2: then
    1/rms is 2^-20 and each of the two Sinkhorn passes divides by 2^40.  A pass hands
    (dc' - sum dc' c') / s back: with c' = 2^-40 after the row pass, every other entry of the
    row gets -2^-40 of u too (the column pass, with c' = 2^-80, gives 2^-80), which is what
    LEAK allows for."""
    T = u.shape[0]
    return dict(dpre=4 * u[:, :S].contiguous(), dpost=2 * u[:, S:2 * S].contiguous(),
                dcomb=2.0 ** 80 * u[:, 2 * S:].reshape(T, S, S).contiguous())


EPS, UNIT_RMS = 2.0 ** 40, 2.0 ** -20
# of |u| < 4 (the nearest values of a product among them), at most 8 entries a row, times W
# or x of at most 4, in dx of one token and in dW of at most 2 * 8 of them
LEAK = 2.0 ** -40 * 4 * 8 * 4 * 16
# Such small terms in one matrix instruction with the leading planes' products: their sum is
# no longer exact, but off by at most a unit in the last place (2^-23, a truncating adder
# included) of the largest product, |c| (1 + 2^-8) at most; the five instructions of the
# lower planes add 2^-8 of that each.
ROUND = 2.0 ** -23 * (1 + 2.0 ** -5)


def rows(T, S, H, seed, f8):
    """As dots, for every row of the weight: a pair of columns each, in a stream each in turn."""
    g = torch.Generator().manual_seed(seed)
    R = (2 + S) * S
    x, w = torch.zeros(T, S, H), torch.zeros(R, S, H)
    want, size = torch.zeros(T, R, dtype=torch.float64), torch.zeros(T, R, dtype=torch.float64)
    at = torch.stack([torch.randperm(H // 2, generator=g)[:S + 2] for _ in range(S)]) * 2
    for r in range(R):
        c, i = r % S, int(at[r % S, r // S])
        a = rand24(g, 1)
        if f8:
            b = torch.ones(T)
            d = (a.double() * 2.0 ** 17).round().float() * 2.0 ** -17
            w[r, c, i], w[r, c, i + 1] = a, d
            x[:, c, i], x[:, c, i + 1] = 1.0, -1.0
            want[:, r] = a.double() - d.double()
        else:
            b = rand24(g, T)
            d, want[:, r] = pair(a, b)
            w[r, c, i], w[r, c, i + 1] = a, 1.0
            x[:, c, i], x[:, c, i + 1] = b, -d
        size[:, r] = (a.double() * b.double()).abs()
    return dict(x=x, w=w.reshape(R, S * H), want=want, size=size)


def streams(T, S, H, seed):
    """dx = dx_in + u W of one row a token (the others have no gradient), x = 0, times 2^-20.
    dx_in is -c of u W."""
    g = torch.Generator().manual_seed(seed)
    R = (2 + S) * S
    w = rand24(g, R, S * H)
    u = torch.zeros(T, R)
    row = torch.randint(0, R, (T,), generator=g)
    v = rand24(g, T)
    u[torch.arange(T), row] = v
    c, want = pair(w[row], v.unsqueeze(1))
    return dict(x=torch.zeros(T, S, H), w=w, **seeds(u, S),
                dx_in=-c.reshape(T, S, H) * UNIT_RMS, want=want.reshape(T, S, H),
                size=c.double().abs().reshape(T, S, H),
                leaks=(row >= 2 * S).double().reshape(T, 1, 1))


def weights(T, S, H, seed, f8):
    """dW of as many rows as there are pairs of neighbouring tokens, each from a pair of its
    own: u x of one token and, with u = 1, -c of the other, times 2^-20.  f8: x is 1.5 and 1,
    and -c, in u, the value next to -1.5 u."""
    g = torch.Generator().manual_seed(seed)
    n, R = S * H, (2 + S) * S
    x, u = torch.zeros(T, n), torch.zeros(T, R)
    want, size = torch.zeros(R, n, dtype=torch.float64), torch.zeros(R, n, dtype=torch.float64)
    pairs = torch.randperm(T // 2, generator=g)[:R] * 2
    for r, t in zip(torch.randperm(R, generator=g).tolist(), pairs.tolist()):
        v = rand24(g, 1)
        if f8:
            x[t], x[t + 1] = 1.5, 1.0
            c, d = pair(v, torch.full((n,), 1.5))
            u[t, r], u[t + 1, r] = v, -c[0]
        else:
            x[t] = rand24(g, n)
            c, d = pair(v, x[t])
            x[t + 1] = -c
            u[t, r], u[t + 1, r] = v, 1.0
        want[r], size[r] = d, c.double().abs()
    return dict(x=x.reshape(T, S, H), **seeds(u, S), want=want, size=size,
                leaks=(torch.arange(R) >= 2 * S).double().unsqueeze(1))


def planes(v, cut=False):
    """Three bf16 parts of fp32 values, in 64 bits: rounded to nearest, or cut."""
    out, rest = [], v.float()
    for _ in range(3):
        if cut:
            p = (rest.view(torch.int32) & -65536).view(torch.float32)
        else:
            p = rest.bfloat16().float()
        out.append(p.double())
        rest = rest - p
    assert not rest.any()
    return out


def product(a, b, cut=False, drop=()):
    """a b as the call forms it: six of the nine products of planes, those in drop left out."""
    pa, pb = planes(a, cut), planes(b, cut)
    return sum(pa[i] * pb[j] for i in range(3) for j in range(3 - i) if (i, j) not in drop)
