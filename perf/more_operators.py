"""Measured cases of the norms around a branch (before it; after it, with its gate and
residual scale, in the post mix) and their gradients, and of the product with 4-bit weights.

``run`` computes a case in plain torch operations, or, where ``own`` is true, through the
package's calls.  Sizes are those of the production site (4 streams of 4096), the wide site
(8 streams of 7168), the 128-wide fixture and odd ones between them.
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # one decoded token's branch input, in the epilogue's 8-bit form, through a projection
        dict(name="q4 token", op="q4", M=1, N=4096, K=4096, group=128, zeros=False, act="q8",
             out="f32", scale="bf16"),
        # a decoded token through an up projection whose groups have zero points of their own
        dict(name="q4 token up", op="q4", M=1, N=16384, K=4096, group=64, zeros=True, act="f32",
             out="f32", scale="f16"),
        # a verify batch of 8 tokens through the same projection
        dict(name="q4 verify", op="q4", M=8, N=16384, K=4096, group=128, zeros=False, act="bf16",
             out="bf16", scale="bf16"),
        # a ragged prompt chunk through the wide site's projection
        dict(name="q4 chunk", op="q4", M=333, N=7168, K=7168, group=128, zeros=True, act="bf16",
             out="f32", scale="bf16"),
        # a short odd chunk's branch input
        dict(name="norm odd", op="norm", T=37, H=1028, z="bf16"),
        # a prefill chunk's branch input
        dict(name="norm prefill", op="norm", T=4096, H=4096, z="bf16"),
        # the gradient of an odd chunk of the wide site, exact input
        dict(name="norm backward wide", op="norm_bwd", T=1001, H=7168, dz="f32", f8=False),
        # a prefill chunk's gradient, its input kept in 8 bits
        dict(name="norm backward prefill", op="norm_bwd", T=4096, H=4096, dz="bf16", f8=True),
        # a decoded token's branch output into the streams, a gate per channel
        dict(name="post token", op="post", T=1, S=4, H=4096, f="f32", gate="channel",
             gate_dtype="f32", gate_act="none"),
        # a prefill chunk, a computed gate per token and channel
        dict(name="post prefill", op="post", T=4096, S=4, H=4096, f="bf16", gate="token",
             gate_dtype="bf16", gate_act="sigmoid"),
        # the fixture's gradient, exact operands
        dict(name="post backward tiny", op="post_bwd", T=4, S=4, H=128, f="f32", f8=False,
             gate="channel", gate_dtype="f32", gate_act="none"),
        # a prefill chunk's gradient, state kept in 8 bits, a computed gate
        dict(name="post backward prefill", op="post_bwd", T=4096, S=4, H=4096, f="bf16", f8=True,
             gate="token", gate_dtype="bf16", gate_act="sigmoid"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["q4", "q4", "q4", "norm", "norm_bwd", "post", "post_bwd"])
    two = ["f32", "bf16"]
    if op == "q4":
        K = _log(rng, 32, 16384, 32)
        N = min(_log(rng, 16, 16384), 67108864 // K)
        M = min(rng.choice([1, 1, _log(rng, 1, 16), _log(rng, 1, 512)]),
                max(1, 17000000000 // (N * K)))
        return dict(op=op, M=M, N=N, K=K, group=rng.choice([32, 64, 128, 128]),
                    zeros=rng.choice([True, False]), act=rng.choice(["f32", "bf16", "q8"]),
                    out=rng.choice(two), scale=rng.choice(["bf16", "f16"]))
    H = _log(rng, 4, 8192, 4)
    if op in ("norm", "norm_bwd"):
        T = min(_log(rng, 1, 8192), 16777216 // H)
        if op == "norm":
            return dict(op=op, T=T, H=H, z=rng.choice(two))
        return dict(op=op, T=T, H=H, dz=rng.choice(two), f8=rng.choice([True, False]))
    S = rng.choice([1, 2, 3, 4, 4, 4, 5, 6, 7, 8, 8])
    T = min(_log(rng, 1, 8192), 67108864 // (S * H))
    case = dict(op=op, T=T, S=S, H=H, f=rng.choice(two),
                gate=rng.choice(["none", "channel", "token", "token"]),
                gate_dtype=rng.choice(two), gate_act=rng.choice(["none", "sigmoid", "silu"]))
    if op == "post_bwd":
        case["f8"] = rng.choice([True, False])
    return case


# ------------------------------------------------------------------ plain forms
def _weight(codes, scales, zeros, group):
    """Codes [N, K/2]: byte j of each 16 holds columns j (low half) and 16 + j of 32."""
    b = codes.unflatten(1, (-1, 16))
    c = torch.cat([b & 15, b >> 4], 2).flatten(1).float()
    at = torch.arange(c.shape[1], device="cuda") // group
    z = 8.0 if zeros is None else zeros.float()[:, at]
    return (c - z) * scales.float()[:, at]


def _plain_q4(s):
    a = s["a"]
    if isinstance(a, tuple):
        a = (a[0].float().unflatten(1, (-1, 32)) * a[1].unsqueeze(2)).flatten(1)
    w = _weight(s["codes"], s["scales"], s["zeros"], s["group"])
    return torch.matmul(a.float(), w.t()).to(s["out"])


def _kept(t, H):
    """Values of an fp32 or bf16 tensor, or of e4m3 codes with an exponent byte per 128."""
    if isinstance(t, tuple):
        e = t[1].int().unsqueeze(-1) - 127
        return torch.ldexp(t[0].float().unflatten(-1, (-1, 128)), e).flatten(-2)[..., :H]
    return t.float()


def _inverse(v):
    return torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    y = s["y"]
    return (y * _inverse(y) * s["nw"]).to(s["z"])


def _plain_norm_bwd(s):
    dz = s["dz"].float()
    y = _kept(s["y"], dz.shape[1])
    r = _inverse(y)
    n, dn = y * r, dz * s["nw"]
    dy = r * (dn - n * (dn * n).mean(1, keepdim=True))
    return dy, (dz * n).sum(0)


def _act(gate, how):
    """The gate's factor and its slope."""
    if gate is None:
        return 1.0, None
    g = gate.float()
    if how is None:
        return g, torch.ones_like(g)
    p = torch.sigmoid(g)
    slope = p * torch.sigmoid(-g)
    return (p, slope) if how == "sigmoid" else (g * p, p + g * slope)


def _plain_post(s):
    x, f, post, comb = s["x"], s["f"].float(), s["post"], s["comb"]
    a, _ = _act(s["gate"], s["gate_act"])
    h = s["alpha"] * a * (f * _inverse(f) * s["nw"])
    mixed = torch.matmul(comb.transpose(1, 2).contiguous(), x)
    return post.unsqueeze(2) * h.unsqueeze(1) + mixed


def _plain_post_bwd(s):
    g, post, comb, nw, alpha = s["g"], s["post"], s["comb"], s["nw"], s["alpha"]
    H = g.shape[2]
    x, f = _kept(s["x"], H), _kept(s["f"], H)
    a, slope = _act(s["gate"], s["gate_act"])
    r = _inverse(f)
    n = f * r
    dx = torch.matmul(comb, g)
    dcomb = torch.matmul(x, g.transpose(1, 2).contiguous())
    dpost = torch.matmul(g, (alpha * a * n * nw).unsqueeze(2)).squeeze(2)
    e = alpha * torch.matmul(post.unsqueeze(1), g).squeeze(1)
    dn = e * a * nw
    df = r * (dn - n * (dn * n).mean(1, keepdim=True))
    dnw = (e * a * n).sum(0)
    if slope is None:
        return dx, df, dpost, dcomb, dnw
    dgate = e * n * nw * slope
    return dx, df, dpost, dcomb, dnw, dgate.sum(0) if s["gate"].dim() == 1 else dgate


# ------------------------------------------------------------------ inputs
_DTYPES = dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)


def _activation(rand, *shape):
    """Unit values with a few loud channels, as a residual stream has them."""
    x = rand(*shape)
    loud = torch.exp(1.5 * rand(shape[-1]).abs()) * (rand(shape[-1]).abs() > 2.0)
    return x * (1 + loud)


def _keep(x):
    """The 8-bit checkpoint of x [..., n]: e4m3 codes, an exponent byte per 128."""
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 128))
    b = x.unflatten(-1, (-1, 128))
    m, p = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0.875, p - 8, p - 9)
    q = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _quantised(rand, N, K, group, zeros, scale):
    """4-bit codes of a random weight, nearest values of each group."""
    G = -(-K // group)
    w = torch.nn.functional.pad(rand(N, K) / math.sqrt(K), (0, G * group - K))
    w = w.unflatten(1, (G, group))
    if zeros:
        lo, hi = w.amin(2).clamp(max=0.0), w.amax(2).clamp(min=0.0)
        scales = ((hi - lo) / 15).to(scale)
        z = torch.round(-lo / scales.float()).clamp(0, 15)
    else:
        scales = (w.abs().amax(2) / 7).to(scale)
        z = torch.full_like(scales, 8.0, dtype=torch.float32)
    c = torch.round(w / scales.float().unsqueeze(2)) + z.unsqueeze(2)
    c = c.clamp(0, 15).to(torch.uint8).flatten(1)[:, :K].unflatten(1, (-1, 2, 16))
    codes = (c[:, :, 0] | (c[:, :, 1] << 4)).flatten(1).contiguous()
    return codes, scales, z.to(torch.uint8) if zeros else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    op = case["op"]
    if op == "q4":
        M, N, K = case["M"], case["N"], case["K"]
        a = _activation(rand, M, K)
        if case["act"] == "q8":
            b = a.unflatten(1, (-1, 32))
            d = b.abs().amax(2) / 127
            a = torch.round(b / d.unsqueeze(2)).clamp(-127, 127).to(torch.int8).flatten(1), d
        else:
            a = a.to(_DTYPES[case["act"]])
        codes, scales, zeros = _quantised(rand, N, K, case["group"], case["zeros"],
                                          _DTYPES[case["scale"]])
        return dict(op=op, a=a, codes=codes, scales=scales, zeros=zeros, group=case["group"],
                    out=_DTYPES[case["out"]])
    T, H = case["T"], case["H"]
    nw = 1 + 0.2 * rand(H)
    if op == "norm":
        return dict(op=op, y=_activation(rand, T, H), nw=nw, z=_DTYPES[case["z"]])
    if op == "norm_bwd":
        y = _activation(rand, T, H)
        return dict(op=op, dz=(rand(T, H) / math.sqrt(T)).to(_DTYPES[case["dz"]]),
                    y=_keep(y) if case["f8"] else y, nw=nw)
    S = case["S"]
    gate = None
    if case["gate"] != "none":
        gate = rand(*((H,) if case["gate"] == "channel" else (T, H)))
        gate = gate.to(_DTYPES[case["gate_dtype"]])
    x, f = _activation(rand, T, S, H), _activation(rand, T, H)
    s = dict(op=op, nw=nw, gate=gate, alpha=0.25,
             gate_act=None if case["gate_act"] == "none" else case["gate_act"],
             post=2 * torch.sigmoid(rand(T, S)), comb=torch.softmax(rand(T, S, S), 2))
    if op == "post":
        return dict(s, x=x, f=f.to(_DTYPES[case["f"]]))
    # the branch output is kept in 8 bits where the state is and it was fp32
    kept = case["f8"] and case["f"] == "f32"
    return dict(s, g=rand(T, S, H) / math.sqrt(T), x=_keep(x) if case["f8"] else x,
                f=_keep(f) if kept else f.to(_DTYPES[case["f"]]))


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    op = s["op"]
    if not own:
        return dict(q4=_plain_q4, norm=_plain_norm, norm_bwd=_plain_norm_bwd, post=_plain_post,
                    post_bwd=_plain_post_bwd)[op](s)
    import mhc_hyper_connection_token_amd as mhc
    if op == "q4":
        return mhc.q4_matmul(s["a"], s["codes"], s["scales"], s["zeros"], dtype=s["out"])
    if op == "norm":
        return mhc.branch_norm(s["y"], s["nw"], EPS, dtype=s["z"])
    if op == "norm_bwd":
        return mhc.branch_norm_bwd(s["dz"], s["y"], s["nw"], EPS)
    how = dict(gate=s["gate"], gate_act=s["gate_act"], alpha=s["alpha"])
    if op == "post":
        return mhc.site_post_norm(s["x"], s["f"], s["nw"], s["post"], s["comb"], EPS, **how)
    out = mhc.site_post_norm_bwd(s["g"], s["x"], s["f"], s["nw"], s["post"], s["comb"], EPS,
                                 **how)
    return out if s["gate"] is not None else out[:5]


_SIZES = dict(f32=4, bf16=2, f16=2)


def work(case):
    op = case["op"]
    if op == "q4":
        M, N, K = case["M"], case["N"], case["K"]
        groups = N * -(-K // case["group"])
        a = M * K * _SIZES[case["act"]] if case["act"] != "q8" else M * K + M * K // 8
        return dict(bytes=N * K // 2 + groups * (3 if case["zeros"] else 2) + a
                    + M * N * _SIZES[case["out"]], flops=2 * M * N * K)
    T, H = case["T"], case["H"]
    if op == "norm":
        return dict(bytes=T * H * (4 + _SIZES[case["z"]]) + 4 * H, flops=4 * T * H)
    if op == "norm_bwd":
        kept = 1 if case["f8"] else 4
        return dict(bytes=T * H * (4 + kept + _SIZES[case["dz"]]) + 8 * H, flops=9 * T * H)
    S = case["S"]
    gate = 0
    if case["gate"] != "none":
        gate = _SIZES[case["gate_dtype"]] * H * (T if case["gate"] == "token" else 1)
    if op == "post":
        return dict(bytes=T * (8 * S * H + _SIZES[case["f"]] * H + 4 * S + 4 * S * S) + gate
                    + 4 * H, flops=2 * T * H * (S * S + S) + 6 * T * H)
    kept = 1 if case["f8"] else 4
    f = 1 if case["f8"] and case["f"] == "f32" else _SIZES[case["f"]]
    dgate = {"none": 0, "channel": 4 * H, "token": 4 * T * H}[case["gate"]]
    return dict(bytes=T * (8 * S * H + kept * S * H + f * H + 4 * H + 8 * (S + S * S)) + gate
                + dgate + 8 * H, flops=4 * T * H * (S * S + S) + 16 * T * H)


# ------------------------------------------------------------------ 64-bit values
def _value64(t, H):
    if not isinstance(t, tuple):
        return t.double()
    codes, scales = t
    size = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"),
                     scales.double() - 127.0)
    return (codes.double() * size.repeat_interleave(128, -1))[..., :H]


def _q4_64(case, s):
    N, K = case["N"], case["K"]
    codes = s["codes"].long().reshape(N, K // 32, 16)
    w = torch.empty(N, K // 32, 32, dtype=torch.float64, device="cuda")
    w[:, :, :16] = codes % 16
    w[:, :, 16:] = codes // 16
    w = w.reshape(N, K)
    wide = s["scales"].double().repeat_interleave(case["group"], 1)[:, :K]
    zero = 8.0 if s["zeros"] is None else \
        s["zeros"].double().repeat_interleave(case["group"], 1)[:, :K]
    w = wide * w - wide * zero
    a = s["a"]
    if case["act"] == "q8":
        a = a[0].double() * a[1].double().repeat_interleave(32, 1)
    return a.double() @ w.t()


def _factor64(gate, how):
    if gate is None:
        return 1.0
    if how is None:
        return gate
    return (1.0 if how == "sigmoid" else gate) / (1 + torch.exp(-gate))


def _branch64(f, nw, gate, how, alpha):
    size = torch.sqrt((f * f).sum(1, keepdim=True) / f.shape[1] + EPS)
    return f / size * nw * _factor64(gate, how) * alpha


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "q4":
        return _q4_64(case, s)
    H = case["H"]
    nw = s["nw"].double()
    if op == "norm":
        return _branch64(s["y"].double(), nw, None, None, 1.0)
    if op == "norm_bwd":
        y, w = _value64(s["y"], H).requires_grad_(), nw.requires_grad_()
        _branch64(y, w, None, None, 1.0).backward(s["dz"].double())
        return y.grad, w.grad
    gate = None if s["gate"] is None else s["gate"].double()
    how, alpha, S = s["gate_act"], s["alpha"], case["S"]
    x, f = _value64(s["x"], H), _value64(s["f"], H)
    post, comb = s["post"].double(), s["comb"].double()
    if op == "post":
        h = _branch64(f, nw, gate, how, alpha)
        return torch.stack([post[:, k, None] * h + sum(comb[:, j, k, None] * x[:, j]
                                                       for j in range(S)) for k in range(S)], 1)
    # the mix's own gradient stream by stream, the branch's by differentiation
    g = s["g"].double()
    dx = torch.stack([sum(comb[:, j, k, None] * g[:, k] for k in range(S))
                      for j in range(S)], 1)
    dcomb = torch.stack([torch.stack([(x[:, j] * g[:, k]).sum(1) for k in range(S)], 1)
                         for j in range(S)], 1)
    leaves = [t.requires_grad_() for t in (f, nw) + (() if gate is None else (gate,))]
    h = _branch64(leaves[0], leaves[1], gate, how, alpha)
    dpost = torch.stack([(g[:, k] * h.detach()).sum(1) for k in range(S)], 1)
    h.backward(sum(post[:, k, None] * g[:, k] for k in range(S)))
    return (dx, f.grad, dpost, dcomb, nw.grad) + (() if gate is None else (gate.grad,))
