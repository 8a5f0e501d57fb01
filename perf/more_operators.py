"""Measured passes of the operators around a layer's QKV projection and its weights' update.

* orthogonalisation of a matrix by Newton-Schulz products, and Muon's update of
  a weight with it (momentum, iteration, decay), weight and momentum in place;
* norm of the queries and keys of each head with the rotation by their position
  in the same pass, between the QKV projection and attention, and its gradient,
  which writes the packed gradient of the projection's output (the values' part
  copied into it) and its maximum for the quantizer.

``run`` computes a pass with elementary torch operations in 32 bits (angles in
64), rounded once at the end; with ``own`` set it makes the framework's calls.
``exact`` gives the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
STEP = (3.4445, -4.7750, 2.0315)     # a, b, c of the Muon optimiser's quintic step
STEPS = 5
NORM_EPS, QK_EPS = 1e-7, 1e-6
BETA, DECAY = 0.95, 0.1
BASE = 10000.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _muon(name, batch, rows, cols, g="bf16", m="fp32", w="bf16", lr=0.02, transposed=False):
    return dict(name=name, op="muon", batch=batch, rows=rows, cols=cols, g=g, m=m, w=w, lr=lr, transposed=transposed)


def _qk(name, op, batch, seq, heads, kv_heads, head_dim, rot, x="bf16", y="bf16", w="bf16", interleaved=False, far=0,
        heads_first=False):
    return dict(name=name, op=op, batch=batch, seq=seq, heads=heads, kv_heads=kv_heads, head_dim=head_dim, rot=rot, x=x,
                y=y, w=w, interleaved=interleaved, far=far, heads_first=heads_first)


def listed():
    return [
        # a low-rank factor of 16 against the benchmark's hidden size: latency
        dict(name="ortho factor", op="ortho", batch=1, rows=16, cols=4096, x="bf16"),
        # per-head matrices, each by itself
        dict(name="ortho heads", op="ortho", batch=32, rows=128, cols=512, x="fp32"),
        # nothing is a multiple of a tile; taller than wide
        dict(name="ortho odd", op="ortho", batch=3, rows=1537, cols=1001, x="bf16"),
        # a small model's projection, master weights in fp32
        _muon("muon small", 1, 1024, 1024, g="fp32", w="fp32", lr=1e-3),
        # the attention-out weight of the benchmark's layer
        _muon("muon square", 1, 4096, 4096),
        # its QKV weight, the three projections each by themselves, bf16 momentum
        _muon("muon qkv", 3, 4096, 4096, m="bf16"),
        # its MLP-up weight, with the gradient as the Wgrad product writes it: [in, out]
        _muon("muon mlp", 1, 16384, 4096, transposed=True),
        # one generated token of 16 sequences deep in their contexts, grouped queries: latency
        _qk("qk token", "qk", 16, 1, 32, 8, 128, 128, far=1 << 20),
        # the benchmark's layer: 31 sequences of 512 tokens, 32 heads of 128
        _qk("qk layer", "qk", 31, 512, 32, 32, 128, 128),
        # half-rotated heads of 80 in neighbouring pairs, fp32, the result's heads ahead of its positions
        _qk("qk odd", "qk", 3, 1999, 16, 16, 80, 40, x="fp32", y="fp32", w="fp32", interleaved=True, heads_first=True),
        # the backward pass on the benchmark's layer
        _qk("qk grad layer", "qk_grad", 31, 512, 32, 32, 128, 128),
        # one long sequence, grouped queries, fp32 weights, an odd number of tokens far from the start
        _qk("qk grad long", "qk_grad", 1, 8191, 32, 8, 128, 64, w="fp32", far=100000, heads_first=True),
    ]


def draw(rng):
    def spread(lo, hi):
        """A whole number between lo and hi, even over the logarithm; odd or even as it falls."""
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["ortho", "muon", "qk", "qk_grad"])
    if op in ("ortho", "muon"):
        while True:
            short, batch = spread(8, 4096), spread(1, 32)
            if rng.random() < 0.5:
                short = -(-short // 64) * 64
            long = short * spread(1, 4) + rng.choice([0, 0, spread(1, 200)])
            if batch * short * short * (3 * long + short) <= 4096 * 4096 * (3 * 16384 + 4096) and batch * short * long <= 1 << 26:
                break
        rows, cols = rng.choice([(short, long), (long, short)])
        if op == "ortho":
            return dict(op=op, batch=batch, rows=rows, cols=cols, x=rng.choice(["bf16", "fp32"]))
        w = rng.choice(["bf16", "fp32"])
        return dict(op=op, batch=batch, rows=rows, cols=cols, g=rng.choice(["bf16", "fp32"]), m=rng.choice(["bf16", "fp32"]),
                    w=w, lr=0.02 if w == "bf16" else 1e-3, transposed=rng.random() < 0.5)
    head_dim = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
    kv_heads = spread(1, 32)
    heads = kv_heads * rng.choice([1, 1, 2, 4, 7])
    tokens = spread(1, min(32768, (1 << 27) // ((heads + 2 * kv_heads) * head_dim)))
    batch = spread(1, min(tokens, 64))
    x = rng.choice(["bf16", "bf16", "fp32"])
    return dict(op=op, batch=batch, seq=max(1, tokens // batch), heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                rot=rng.choice([head_dim, head_dim, head_dim // 2]), x=x, y=rng.choice(["bf16", x]),
                w=rng.choice(["bf16", "fp32"]), interleaved=rng.random() < 0.3, far=rng.choice([0, 0, 5000, 1 << 20]),
                heads_first=rng.random() < 0.5)


def work(case):
    """Bytes and operations of one pass; of a symmetric product one half is counted."""
    size = {"bf16": 2, "fp32": 4}
    if case["op"] in ("ortho", "muon"):
        b, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        flops = STEPS * b * m * m * (3 * n + m)
        if case["op"] == "ortho":
            return dict(bytes=b * m * n * (size[case["x"]] + 2), flops=flops)
        return dict(bytes=b * m * n * (size[case["g"]] + 2 * size[case["m"]] + 2 * size[case["w"]]), flops=flops)
    t, d = case["batch"] * case["seq"], case["head_dim"]
    heads, kv, bx, by = case["heads"], case["kv_heads"], size[case["x"]], size[case["y"]]
    n = t * (heads + kv) * d
    if case["op"] == "qk":
        return dict(bytes=n * (bx + by) + 2 * d * size[case["w"]] + 8 * t, flops=9 * n)
    return dict(bytes=n * (2 * bx + by) + t * kv * d * (bx + by) + 2 * d * (size[case["w"]] + 4) + 8 * t, flops=18 * n)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["op"] in ("ortho", "muon"):
        b, r, c = case["batch"], case["rows"], case["cols"]
        # a linear layer's gradient: a few directions stand far out of the noise of the rest
        k = min(8, r, c)
        u, v = normal(b, r, k) * 0.6 ** torch.arange(k, device="cuda"), normal(b, k, c)

        def gradient(mix):
            return 1e-3 * (0.1 * normal(b, r, c) + torch.stack([p @ q for p, q in zip(u * mix, v)]))

        if case["op"] == "ortho":
            x = gradient(1.0).to(TYPES[case["x"]])
            return dict(case=case, x=x)
        g = gradient(0.7 + 0.3 * normal(b, 1, k)).to(TYPES[case["g"]])
        if case["transposed"]:
            g = g.transpose(1, 2).contiguous()
        return dict(case=case, grad=g, momentum=gradient(1.0).to(TYPES[case["m"]]),
                    w=(0.02 * normal(b, r, c)).to(TYPES[case["w"]]))

    b, s, h, kv, d = (case[k] for k in ("batch", "seq", "heads", "kv_heads", "head_dim"))
    # the projection's output, packed: queries, keys, values; some channels of the queries and keys stand out
    scale = torch.where(torch.rand((h + 2 * kv) * d, device="cuda", generator=gen) < 0.03, 8.0, 1.0)
    qkv = (normal(b, s, (h + 2 * kv) * d) * scale).to(TYPES[case["x"]])
    start = torch.randint(0, case["far"] + 1, (b, 1), device="cuda", generator=gen)
    state = dict(case=case, qkv=qkv, positions=start + torch.arange(s, device="cuda"),
                 qw=(1 + 0.2 * normal(d)).to(TYPES[case["w"]]), kw=(1 + 0.2 * normal(d)).to(TYPES[case["w"]]))
    # f_i = BASE^(-2 i / rot), in 64 bits
    state["freqs"] = torch.tensor([BASE ** (-2 * i / case["rot"]) for i in range(case["rot"] // 2)],
                                  dtype=torch.float64, device="cuda")
    if case["op"] == "qk_grad":
        for name, n in (("dq", h), ("dk", kv), ("dv", kv)):
            shape = (b, n, s, d) if case["heads_first"] else (b, s, n, d)
            state[name] = (1e-3 * normal(*shape)).to(TYPES[case["y"]])
    return state


def _heads(case, state):
    """The queries, keys and values of the packed projection, [batch, seq, heads, head_dim]."""
    h, kv, d = case["heads"], case["kv_heads"], case["head_dim"]
    t = state["qkv"].unflatten(2, (h + 2 * kv, d))
    return t[:, :, :h], t[:, :, h:h + kv], t[:, :, h + kv:]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return (_framework if own else _plain)(case["op"], case, state)


def _framework(op, case, s):
    from precision_block_scaled_amd import pipeline as PL
    if op == "ortho":
        return dict(y=PL.orthogonalize(s["x"], coefficients=(STEP,) * STEPS, eps=NORM_EPS))
    if op == "muon":
        grad = s["grad"].transpose(1, 2) if case["transposed"] else s["grad"]
        PL.muon(s["w"], s["momentum"], grad, case["lr"], beta=BETA, weight_decay=DECAY, coefficients=(STEP,) * STEPS,
                eps=NORM_EPS)
        return dict(w=s["w"], momentum=s["momentum"])
    q, k, _ = _heads(case, s)
    rest = dict(freqs=s["freqs"], interleaved=case["interleaved"], eps=QK_EPS)
    if op == "qk":
        outs = {}
        if case["heads_first"]:
            outs = {n: torch.empty(t.transpose(1, 2).shape, dtype=TYPES[case["y"]], device=t.device).transpose(1, 2)
                    for n, t in (("q_out", q), ("k_out", k))}
        yq, yk = PL.qk_norm_rope(q, k, s["qw"], s["kw"], s["positions"], out_dtype=TYPES[case["y"]], **rest, **outs)
        return dict(q=yq.transpose(1, 2), k=yk.transpose(1, 2)) if case["heads_first"] else dict(q=yq, k=yk)
    dq, dk, dv = ((s[n].transpose(1, 2) if case["heads_first"] else s[n]) for n in ("dq", "dk", "dv"))
    out, amax = torch.empty_like(s["qkv"]), torch.empty(1, device=dq.device)
    oq, ok, ov = _heads(case, dict(qkv=out))
    _, _, dqw, dkw = PL.qk_norm_rope_grad(dq, dk, q, k, s["qw"], s["kw"], s["positions"], dv=dv, dq_out=oq, dk_out=ok,
                                          dv_out=ov, amax=amax, **rest)
    return dict(dqkv=out, dqw=dqw, dkw=dkw, amax=amax.to(out.dtype))


def _newton_schulz(x):
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NORM_EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    a, b, c = STEP
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2) if tall else x


def _turn(x, cos, sin, rot, interleaved):
    """Turns the pairs of the first `rot` of the last axis."""
    if interleaved:
        p, q = x[..., :rot:2], x[..., 1:rot:2]
        pairs = torch.stack((p * cos - q * sin, q * cos + p * sin), -1).flatten(-2)
    else:
        p, q = x[..., :rot // 2], x[..., rot // 2:rot]
        pairs = torch.cat((p * cos - q * sin, q * cos + p * sin), -1)
    return torch.cat((pairs, x[..., rot:]), -1)


def _plain(op, case, s):
    if op == "ortho":
        return dict(y=_newton_schulz(s["x"].float()).contiguous().bfloat16())
    if op == "muon":
        grad = (s["grad"].transpose(1, 2) if case["transposed"] else s["grad"]).float()
        m = BETA * s["momentum"].float() + (1 - BETA) * grad
        step = case["lr"] * max(1.0, case["rows"] / case["cols"]) ** 0.5
        o = _newton_schulz(BETA * m + (1 - BETA) * grad)
        s["w"].copy_((1 - case["lr"] * DECAY) * s["w"].float() - step * o)
        s["momentum"].copy_(m)
        return dict(w=s["w"], momentum=s["momentum"])
    q, k, v = _heads(case, s)
    rot, inter = case["rot"], case["interleaved"]
    angle = s["positions"].double()[:, :, None, None] * s["freqs"]
    cos, sin = angle.cos().float(), angle.sin().float()

    def rows(t):
        t = t.float()
        r = 1 / (t.square().mean(-1, keepdim=True) + QK_EPS).sqrt()
        return t * r, r

    if op == "qk":
        def forward(t, w):
            y = _turn(rows(t)[0] * w.float(), cos, sin, rot, inter).to(TYPES[case["y"]])
            return y.transpose(1, 2).contiguous() if case["heads_first"] else y
        return dict(q=forward(q, s["qw"]), k=forward(k, s["kw"]))

    def backward(dy, t, w):
        g = _turn(dy.float(), cos, -sin, rot, inter)
        n, r = rows(t)
        u = g * w.float()
        return r * (u - n * (u * n).mean(-1, keepdim=True)), (g * n).sum((0, 1, 2))

    dq, dk, dv = ((s[n].transpose(1, 2) if case["heads_first"] else s[n]) for n in ("dq", "dk", "dv"))
    gq, dqw = backward(dq, q, s["qw"])
    gk, dkw = backward(dk, k, s["kw"])
    out = torch.cat((gq, gk, dv.float()), 2).to(s["qkv"].dtype).flatten(2)
    return dict(dqkv=out, dqw=dqw, dkw=dkw, amax=out.abs().amax().reshape(1))


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def _orthogonal64(x):
    """x over its Frobenius norm, multiplied in each step by the step's polynomial of its smaller Gram matrix."""
    x = x.double()
    x = x / (torch.linalg.matrix_norm(x) + NORM_EPS)
    wide = x if x.shape[0] <= x.shape[1] else x.t()
    for _ in range(STEPS):
        gram = wide.mm(wide.t())
        poly = torch.addmm(gram, gram, gram, beta=STEP[1], alpha=STEP[2])
        poly.diagonal().add_(STEP[0])
        wide = poly.mm(wide)
    return wide if x.shape[0] <= x.shape[1] else wide.t()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ortho":
        return dict(y=torch.stack([_orthogonal64(x) for x in s["x"]]))
    if op == "muon":
        w, momentum = s["w"].double(), s["momentum"].double()
        for i in range(case["batch"]):
            g = (s["grad"][i].t() if case["transposed"] else s["grad"][i]).double()
            momentum[i].lerp_(g, 1 - BETA)
            update = _orthogonal64(momentum[i].lerp(g, 1 - BETA))
            w[i].mul_(1 - case["lr"] * DECAY)
            w[i].sub_(update, alpha=case["lr"] * math.sqrt(max(1.0, case["rows"] / case["cols"])))
        return dict(w=w, momentum=momentum)

    rot, h, kv = case["rot"], case["heads"], case["kv_heads"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, :, None, None] * s["freqs"])
    qkv = s["qkv"].double().unflatten(2, (h + 2 * kv, case["head_dim"]))
    grads = op == "qk_grad"
    ys, leaves = [], []
    for part, w in ((qkv[:, :, :h], s["qw"]), (qkv[:, :, h:h + kv], s["kw"])):
        x, w = part.clone().requires_grad_(grads), w.double().requires_grad_(grads)
        u = torch.nn.functional.rms_norm(x, x.shape[-1:], w, QK_EPS)
        head = u[..., :rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        if not case["interleaved"]:
            head = head.transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
        if not case["interleaved"]:
            turned = turned.transpose(-1, -2)
        ys.append(torch.cat((turned.flatten(-2), u[..., rot:]), -1))
        leaves += [x, w]
    if not grads:
        return {n: y.transpose(1, 2) if case["heads_first"] else y for n, y in zip("qk", ys)}
    dq, dk, dv = ((s[n].transpose(1, 2) if case["heads_first"] else s[n]).double() for n in ("dq", "dk", "dv"))
    gq, dqw, gk, dkw = torch.autograd.grad(ys, leaves, (dq, dk))
    out = torch.cat((gq, gk, dv), 2).flatten(2)
    return dict(dqkv=out, dqw=dqw, dkw=dkw, amax=out.abs().amax().reshape(1))
