"""Measured cases of the 8-bit and backward operators: block encoding, 8-bit
matrix product, and the backward passes of a site's two halves.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
through the package's calls.  Sizes are those of the production site (4 streams
of 4096), the wide site (8 streams of 7168), the 128-wide fixture and odd ones
between them.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0


def listed():
    return [
        # one decoded token's branch input, encoded for the branch's product
        dict(name="encode token", op="encode", mode="rows", rows=1, cols=4096, dtype="f32"),
        # the stream state of a prefill chunk (4096 tokens x 4 streams), kept for the backward pass
        dict(name="encode state", op="encode", mode="rows", rows=16384, cols=4096, dtype="f32"),
        # an output gradient of an odd batch, needed along both axes (input and weight gradient)
        dict(name="encode gradient both ways", op="encode", mode="both", rows=1001, cols=7168,
             dtype="bf16"),
        # a decoded token through a square projection
        dict(name="matmul decode", op="matmul", M=1, N=4096, K=4096, square=True, dtype="f32"),
        # a verify batch through an up projection, bf16 out
        dict(name="matmul verify", op="matmul", M=8, N=16384, K=4096, square=True, dtype="bf16"),
        # a ragged chunk through the wide site's projection
        dict(name="matmul ragged", op="matmul", M=333, N=7168, K=7168, square=True, dtype="f32"),
        # a prefill chunk through an up projection
        dict(name="matmul prefill", op="matmul", M=4096, N=16384, K=4096, square=True,
             dtype="f32"),
        # a weight gradient: tokens are the summed axis, both sides scaled along it
        dict(name="matmul weight gradient", op="matmul", M=7168, N=4096, K=1024, square=False,
             dtype="f32"),
        # the 128-wide fixture's backward, exact (fp32) operands
        dict(name="post backward tiny", op="post_bwd", T=4, S=4, H=128, f8=False),
        # a prefill chunk's post half, state and branch output kept in 8 bits
        dict(name="post backward prefill", op="post_bwd", T=4096, S=4, H=4096, f8=True),
        # a short odd chunk, exact operands
        dict(name="pre backward odd", op="pre_bwd", T=37, S=3, H=1028, iters=20, f8=False),
        # a prefill chunk's pre half from the kept state
        dict(name="pre backward prefill", op="pre_bwd", T=4096, S=4, H=4096, iters=20, f8=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["encode", "matmul", "matmul", "post_bwd", "pre_bwd"])
    if op == "encode":
        cols = _log(rng, 4, 16384, 4)
        rows = min(_log(rng, 1, 16384), 67108864 // cols)
        return dict(op=op, mode=rng.choice(["rows", "both", "square", "repack"]), rows=rows,
                    cols=cols, dtype=rng.choice(["f32", "bf16"]))
    if op == "matmul":
        K = _log(rng, 128, 16384, 128)
        N = _log(rng, 4, 16384, 4)
        M = min(_log(rng, 1, 8192), max(1, 274877906944 // (K * N)))
        return dict(op=op, M=M, N=N, K=K, square=rng.choice([True, True, False]),
                    dtype=rng.choice(["f32", "bf16"]))
    S = rng.choice([1, 2, 3, 4, 4, 4, 5, 6, 7, 8, 8])
    H = _log(rng, 4, 8192, 4)
    T = min(_log(rng, 1, 8192), 33554432 // (S * H))
    case = dict(op=op, T=T, S=S, H=H, f8=rng.choice([True, True, False]))
    if op == "pre_bwd":
        case["iters"] = rng.choice([1, 3, 20, 20, 20, 33])
    return case


def _up(n):
    return -(-n // BLOCK) * BLOCK


# ------------------------------------------------------------------ plain forms
def _encode(x):
    """x [..., n] -> e4m3 codes [..., n up to 128] and one exponent byte per block."""
    x = torch.nn.functional.pad(x.float(), (0, _up(x.shape[-1]) - x.shape[-1]))
    b = x.unflatten(-1, (-1, BLOCK))
    a = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
    return _codes(b, a)


def _codes(b, a):
    m, p = torch.frexp(a)
    e = torch.where(m > 0.875, p - 8, p - 9)
    e = torch.where(a > 0, e.clamp(min=-126), 0)
    q = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _encode_square(x):
    """x [n, k] -> codes [n, k up to 128], one exponent byte per 128 x 128 square."""
    n, k = x.shape
    x = torch.nn.functional.pad(x.float(), (0, _up(k) - k, 0, _up(n) - n))
    b = x.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))  # [nb, 128, kb, 128]
    a = torch.where(torch.isfinite(b), b.abs(), 0.0).amax((1, 3))
    q, e = _codes(b, a.unsqueeze(1).expand(-1, BLOCK, -1))
    return q.reshape(x.shape)[:n].contiguous(), e[:, 0].contiguous()


def _decode(codes, scales):
    """Values of codes [..., n] with an exponent byte per 128 (of each row)."""
    e = scales.int().unsqueeze(-1) - 127
    return torch.ldexp(codes.float().unflatten(-1, (-1, BLOCK)), e).flatten(-2)


def _operand(codes, scales):
    if scales.shape[0] != codes.shape[0]:
        scales = scales.repeat_interleave(BLOCK, 0)[:codes.shape[0]]
    return _decode(codes, scales)


def _plain_encode(s):
    if s["mode"] == "rows":
        return _encode(s["x"])
    if s["mode"] == "both":
        return _encode(s["x"]) + _encode(s["x"].t())
    if s["mode"] == "square":
        return _encode_square(s["x"]) + _encode_square(s["x"].t())
    return _encode(_decode(s["codes"], s["scales"])[:, :s["cols"]].t())


def _plain_matmul(s):
    out = torch.matmul(_operand(s["a"], s["a_scales"]), _operand(s["b"], s["b_scales"]).t())
    return out.to(s["dtype"])


def _kept(t, H):
    return _decode(*t)[..., :H] if isinstance(t, tuple) else t


def _plain_post_bwd(s):
    g, post, comb = s["g"], s["post"], s["comb"]
    x, f = _kept(s["x"], g.shape[2]), _kept(s["f"], g.shape[2])
    dx = torch.matmul(comb, g)
    df = torch.matmul(post.unsqueeze(1), g).squeeze(1)
    dpost = torch.matmul(g, f.unsqueeze(2)).squeeze(2)
    dcomb = torch.matmul(x, g.transpose(1, 2).contiguous())
    return dx, df, dpost, dcomb


def _plain_pre_bwd(s):
    w, scale, base, dy = s["w"], s["scale"], s["base"], s["dy"]
    T, S, H = s["dx_in"].shape
    n = S * H
    x = _kept(s["x"], H)
    flat = x.reshape(T, n)
    raw = torch.matmul(flat, w.t())
    rinv = torch.rsqrt(flat.square().mean(1, keepdim=True) + s["eps"])
    m = raw * rinv
    group = s["group"]
    z = scale[group] * m + base
    pre, half = torch.sigmoid(z[:, :S]), torch.sigmoid(z[:, S:2 * S])
    c0 = torch.exp(z[:, 2 * S:]).reshape(T, S, S)
    c, kept = c0, []
    for axis in (2, 1) * s["iters"]:
        total = c.sum(axis, keepdim=True) + s["eps"]
        c = c / total
        kept.append((c, total, axis))
    dc = s["dcomb"]
    for c, total, axis in reversed(kept):
        dc = (dc - (dc * c).sum(axis, keepdim=True)) / total
    dpre = s["dpre"] + torch.matmul(x, dy.unsqueeze(2)).squeeze(2)
    dz = torch.cat([dpre * pre * (1 - pre), s["dpost"] * 2 * half * (1 - half),
                    (dc * c0).reshape(T, S * S)], 1)
    dm = scale[group] * dz
    u = dm * rinv
    alpha = -(dm * m).sum(1, keepdim=True) * rinv.square() / n
    dx = s["dx_in"] + pre.unsqueeze(2) * dy.unsqueeze(1)
    dx = dx + (torch.matmul(u, w) + alpha * flat).reshape(T, S, H)
    dw = torch.matmul(u.t().contiguous(), flat)
    dscale = torch.zeros_like(scale).index_add_(0, group, (dz * m).sum(0))
    return dx, dw, dscale, dz.sum(0)


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _activation(rand, *shape):
    """Unit values with a few loud channels, as a residual stream has them."""
    x = rand(*shape)
    loud = torch.exp(1.5 * rand(shape[-1]).abs()) * (rand(shape[-1]).abs() > 2.0)
    return x * (1 + loud)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    op = case["op"]
    if op == "encode":
        x = _activation(rand, case["rows"], case["cols"]).to(_dtype(case))
        s = dict(op=op, mode=case["mode"], x=x, cols=case["cols"])
        if case["mode"] == "repack":
            s["codes"], s["scales"] = _encode(x)
        return s
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        a, a_scales = _encode(_activation(rand, M, K))
        b, b_scales = (_encode_square if case["square"] else _encode)(rand(N, K) / math.sqrt(K))
        return dict(op=op, a=a, a_scales=a_scales, b=b, b_scales=b_scales,
                    square=case["square"], dtype=_dtype(case))
    T, S, H = case["T"], case["S"], case["H"]

    def keep(t):
        return _encode(t) if case["f8"] else t

    x = keep(_activation(rand, T, S, H))
    if op == "post_bwd":
        comb = torch.softmax(rand(T, S, S), 2)
        return dict(op=op, g=rand(T, S, H) / math.sqrt(T), x=x, f=keep(_activation(rand, T, H)),
                    post=2 * torch.sigmoid(rand(T, S)), comb=comb)
    R = (2 + S) * S
    group = torch.tensor([0] * S + [1] * S + [2] * (S * S), device="cuda")
    return dict(op=op, x=x, w=rand(R, S * H) / math.sqrt(S * H),
                scale=0.5 + rand(3).abs().clamp(max=1.0), base=rand(R) * 0.3, group=group,
                dy=rand(T, H) / math.sqrt(T), dpre=rand(T, S), dpost=rand(T, S),
                dcomb=rand(T, S, S), dx_in=rand(T, S, H) / math.sqrt(T), iters=case["iters"],
                eps=1e-6)


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    op = s["op"]
    if not own:
        return dict(encode=_plain_encode, matmul=_plain_matmul, post_bwd=_plain_post_bwd,
                    pre_bwd=_plain_pre_bwd)[op](s)
    import mhc_hyper_connection_token_amd as mhc
    if op == "encode":
        if s["mode"] == "repack":
            return mhc.f8_repack(s["codes"], s["scales"], s["cols"])
        return mhc.f8_encode(s["x"], transposed=s["mode"] != "rows", square=s["mode"] == "square")
    if op == "matmul":
        return mhc.f8_matmul(s["a"], s["a_scales"], s["b"], s["b_scales"], dtype=s["dtype"])
    if op == "post_bwd":
        return mhc.site_post_bwd(s["g"], s["x"], s["f"], s["post"], s["comb"])
    return mhc.site_pre_bwd(s["x"], s["w"], s["scale"], s["base"], s["iters"], s["eps"], s["dy"],
                            s["dpost"], s["dcomb"], dpre=s["dpre"], dx_in=s["dx_in"])


def work(case):
    op = case["op"]
    if op == "encode":
        n = case["rows"] * case["cols"]
        size = 1 if case["mode"] == "repack" else 4 if case["dtype"] == "f32" else 2
        outs = 2 if case["mode"] in ("both", "square") else 1
        return dict(bytes=n * (size + outs), flops=2 * n)
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=M * K + N * K + M * N * size, flops=2 * M * N * K)
    T, S, H = case["T"], case["S"], case["H"]
    kept = 1 if case["f8"] else 4
    if op == "post_bwd":
        return dict(bytes=T * (8 * S * H + kept * S * H + kept * H + 4 * H + 8 * (S + S * S)),
                    flops=4 * T * H * (S * S + S))
    R = (2 + S) * S
    return dict(bytes=T * (8 * S * H + kept * S * H + 4 * H + 4 * (2 * S + S * S)) + 8 * R * S * H,
                flops=6 * T * R * S * H + 6 * T * S * H)


# ------------------------------------------------------------------ 64-bit values
def _value64(codes, exponents):
    """Codes times two to their block's exponent, in 64 bits, blocks of 128 per row."""
    width = codes.shape[-1]
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"),
                      exponents.double() - 127.0)
    return codes.double() * scale.repeat_interleave(BLOCK, -1)[..., :width]


def _grid64(v):
    """Nearest e4m3 value of v (ties to the even mantissa), NaN where v is not finite."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.where(torch.isfinite(v), torch.round(v / step) * step, math.nan)


def _blocks64(x, tall):
    """The definition, block by block: tall = rows of x per block (1 or 128)."""
    n, k = x.shape
    full = torch.zeros(-(-n // tall) * tall, _up(k), dtype=torch.float64, device="cuda")
    full[:n, :k] = x.double()
    size = torch.where(torch.isfinite(full), full.abs(), 0.0)
    size = size.reshape(-1, tall, _up(k) // BLOCK, BLOCK).amax((1, 3))
    e = torch.ceil(torch.log2(size.clamp(min=1e-60) / E4M3_MAX))
    e = torch.where(size > torch.exp2(e) * E4M3_MAX, e + 1, e)
    e = torch.where(size <= torch.exp2(e - 1) * E4M3_MAX, e - 1, e)
    e = torch.where(size > 0, e.clamp(min=-126.0), 0.0)
    wide = e.repeat_interleave(tall, 0)[:n].repeat_interleave(BLOCK, 1)
    return _grid64(full[:n] / torch.exp2(wide)), e + 127


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "encode":
        if case["mode"] == "repack":
            x = _value64(s["codes"], s["scales"])[:, :case["cols"]]
            return _blocks64(x.t(), 1)[0], None
        tall = BLOCK if case["mode"] == "square" else 1
        found = (_blocks64(s["x"], tall)[0], None)
        return found if case["mode"] == "rows" else found + (_blocks64(s["x"].t(), tall)[0], None)
    if op == "matmul":
        b_scales = s["b_scales"]
        if case["square"]:
            b_scales = b_scales[torch.arange(case["N"], device="cuda") // BLOCK]
        return _value64(s["a"], s["a_scales"]) @ _value64(s["b"], b_scales).t()
    H = case["H"]
    x, f = (t if t is None else (_value64(*t)[..., :H] if case["f8"] else t.double())
            for t in (s["x"], s.get("f")))
    if op == "post_bwd":
        leaves = [t.requires_grad_() for t in (x, f, s["post"].double(), s["comb"].double())]
        x, f, post, comb = leaves
        out = post[:, :, None] * f[:, None] + torch.matmul(comb.transpose(1, 2), x)
        out.backward(s["g"].double())
        return x.grad, f.grad, post.grad, comb.grad
    S = case["S"]
    leaves = [t.requires_grad_() for t in (x, s["w"].double(), s["scale"].double(),
                                           s["base"].double())]
    x, w, scale, base = leaves
    flat = x.flatten(1)
    mixes = (flat @ w.t()) / torch.sqrt((flat * flat).mean(1, keepdim=True) + s["eps"])
    parts = [mixes[:, :S] * scale[0], mixes[:, S:2 * S] * scale[1], mixes[:, 2 * S:] * scale[2]]
    z_pre, z_post, z_comb = torch.split(torch.cat(parts, 1) + base, [S, S, S * S], 1)
    pre, post = 1 / (1 + torch.exp(-z_pre)), 2 / (1 + torch.exp(-z_post))
    comb = torch.exp(z_comb).unflatten(1, (S, S))
    for _ in range(case["iters"]):
        comb = comb / (comb.sum(2, keepdim=True) + s["eps"])
        comb = comb / (comb.sum(1, keepdim=True) + s["eps"])
    y = (pre[:, :, None] * x).sum(1)
    torch.autograd.backward([y, pre, post, comb], [s[k].double() for k in
                                                   ("dy", "dpre", "dpost", "dcomb")])
    return x.grad + s["dx_in"].double(), w.grad, scale.grad, base.grad
