"""Measured passes of the operators at the two ends of a training step's linear layers.

* layer norm, whose output is what the quantized linears read, and its
  gradient (dx, and the weight's and bias's gradients summed over the rows);
* softmax cross entropy of a linear head over a large vocabulary, from the
  hidden states and the head's weight, without keeping the logits, and its
  gradient (dx and dw);
* distillation through the same head: the Kullback-Leibler divergence from a
  teacher's softmax over its k highest logits to the student's softmax over the
  whole vocabulary, and its gradient.

``run`` computes a pass with elementary torch operations in 32 bits, rounded
once at the end; with ``own`` set it makes the framework's calls.  ``exact``
gives the same outputs in 64 bits from torch's own definitions and autograd.
"""
import math

import torch

own = False

IGNORE = -100            # target of a row that takes no part in the loss
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # layer norm ahead of a linear layer: a handful of rows (one generated token of 16 sequences),
        # where the call itself is what counts
        dict(name="norm 16 rows", op="norm", rows=16, cols=4096, x="bf16", y="bf16", w="bf16", amax=False),
        # the norm ahead of the QKV projection of the benchmark's layer (31 x 512 tokens, hidden 4096),
        # which hands the quantizer max |y|
        dict(name="norm layer", op="norm", rows=15872, cols=4096, x="bf16", y="bf16", w="bf16", amax=True),
        # an fp32 residual stream normalised into the bf16 tensor that the quantizer reads, wide rows
        dict(name="norm wide", op="norm", rows=8192, cols=16384, x="fp32", y="bf16", w="fp32", amax=True),
        # its backward pass on the benchmark's layer
        dict(name="norm grad layer", op="norm_grad", rows=15872, cols=4096, x="bf16", y="bf16", w="bf16"),
        # an odd width in fp32: rows that start at any 4-byte address
        dict(name="norm grad odd", op="norm_grad", rows=4099, cols=1537, x="fp32", y="fp32", w="fp32"),
        # a short evaluation sequence against a small vocabulary: latency
        dict(name="xent small", op="xent", tokens=61, vocab=1021, hidden=512, ignored=0.0),
        # scoring a batch: losses only
        dict(name="xent batch", op="xent", tokens=4096, vocab=32768, hidden=4096, ignored=0.0),
        # fine-tuning step with the prompt's tokens masked out; nothing is a multiple of a tile
        dict(name="xent step masked", op="xent_grad", tokens=2047, vocab=49999, hidden=2048, ignored=0.3),
        # pre-training step: one sequence of 8192 tokens, a vocabulary of 131072
        dict(name="xent step", op="xent_grad", tokens=8192, vocab=131072, hidden=4096, ignored=0.0),
        # distillation losses against 64 stored teacher logits per token
        dict(name="distill batch", op="distill", tokens=2048, vocab=65536, hidden=4096, top=64, tau=1.0, ignored=0.0),
        # a distillation step with padded rows and padded slots
        dict(name="distill step", op="distill_grad", tokens=4096, vocab=32768, hidden=2048, top=32, tau=2.0, ignored=0.1),
        # a tiny one
        dict(name="distill small", op="distill_grad", tokens=37, vocab=2003, hidden=256, top=7, tau=1.5, ignored=0.1),
    ]


def draw(rng):
    def spread(lo, hi):
        """A whole number between lo and hi, even over the logarithm; odd or even as it falls."""
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "norm_grad", "xent", "xent_grad", "distill", "distill_grad"])
    if op.startswith("norm"):
        cols = spread(8, 16384)
        if rng.random() < 0.5:
            cols = -(-cols // 64) * 64
        case = dict(op=op, rows=spread(1, min(65536, (1 << 27) // cols)), cols=cols, x=rng.choice(["bf16", "fp32"]),
                    y="bf16", w=rng.choice(["bf16", "fp32"]))
        if case["x"] == "fp32" and rng.random() < 0.5:
            case["y"] = "fp32"
        if op == "norm":
            case["amax"] = rng.random() < 0.5
        return case
    while True:
        case = dict(op=op, tokens=spread(1, 8192), vocab=spread(128, 131072), hidden=64 * spread(1, 64),
                    ignored=rng.choice([0.0, 0.0, 0.2, 0.6]))
        if case["tokens"] * case["vocab"] * case["hidden"] <= 1 << 41:
            break
    if op.startswith("distill"):
        case["top"] = min(spread(1, 128), case["vocab"])
        case["tau"] = rng.choice([1.0, 2.0, 0.7])
    return case


def work(case):
    """Bytes and operations of one pass.  The losses' gradient passes form the
    logits twice, since the loss does not keep them: 2 products for the loss
    and the recomputation and 2 for dx and dw."""
    if case["op"].startswith("norm"):
        n, c = case["rows"], case["cols"]
        bx, by, bw = (2 if case[k] == "bf16" else 4 for k in ("x", "y", "w"))
        if case["op"] == "norm":
            return dict(bytes=n * c * (bx + by) + 2 * c * bw + 8 * n, flops=8 * n * c)
        return dict(bytes=n * c * (2 * bx + by) + c * (bw + 8) + 8 * n, flops=14 * n * c)
    t, v, h = case["tokens"], case["vocab"], case["hidden"]
    live = max(1, t - int(t * case["ignored"]))
    slots = 12 * case["top"] if "top" in case else 8
    if case["op"].endswith("_grad"):
        return dict(bytes=4 * (t * h + v * h) + t * (slots + 12), flops=8 * live * v * h)
    return dict(bytes=2 * (t * h + v * h) + t * (slots + 8), flops=2 * live * v * h)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    if case["op"].startswith("norm"):
        n, c = case["rows"], case["cols"]
        # activations with a few outlier channels, as in the benchmark's inputs
        scale = torch.where(uniform(c) < 8 / max(c, 64), 20.0, 1.0)
        x = (normal(n, c) * scale + 0.1 * normal(c)).to(TYPES[case["x"]])
        gamma = (1 + 0.2 * normal(c)).to(TYPES[case["w"]])
        beta = (0.1 * normal(c)).to(TYPES[case["w"]])
        state = dict(case=case, x=x, gamma=gamma, beta=beta)
        if case["op"] == "norm_grad":
            x64 = x.double()
            mean = x64.mean(1)
            state["mean"] = mean.float()
            state["rstd"] = ((x64 - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
            state["dy"] = (1e-3 * normal(n, c)).to(TYPES[case["y"]])
        return state

    t, v, h = case["tokens"], case["vocab"], case["hidden"]
    w = (0.02 * normal(v, h)).bfloat16()
    ids = torch.randint(0, v, (t,), device="cuda", generator=g)
    # hidden states that know their target: its logit stands out by 0 to 10
    lift = 10 * uniform(t, 1) / (0.02 ** 2 * h)
    x = (normal(t, h) + lift * w[ids].float()).bfloat16()
    live = torch.arange(t, device="cuda") >= int(t * case["ignored"])
    live = live[torch.randperm(t, device="cuda", generator=g)]
    state = dict(case=case, x=x, w=w)
    if case["op"].startswith("xent"):
        state["targets"] = torch.where(live, ids, IGNORE)
    else:
        k = case["top"]
        # k different entries of each row, the target first: an arithmetic walk through the vocabulary
        step = torch.randint(1, max(2, v // k), (t, 1), device="cuda", generator=g)
        top = (ids[:, None] + step * torch.arange(k, device="cuda")) % v
        logits = (2 * normal(t, k)).sort(1, descending=True).values
        logits[:, 0] += 4 * uniform(t)
        # some rows hold fewer entries than slots: the rest is marked -1, whatever logit stands there
        held = torch.randint(1, k + 1, (t, 1), device="cuda", generator=g)
        held = torch.where(uniform(t, 1) < 0.2, held, k)
        held = torch.where(live[:, None], held, 0)
        state["top_ids"] = torch.where(torch.arange(k, device="cuda") < held, top, -1)
        state["top_logits"] = logits
    if case["op"].endswith("_grad"):
        # weights of the tokens in a mean over the live ones
        state["dloss"] = (0.5 + uniform(t)) / max(1, t - int(t * case["ignored"]))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return (_framework if own else _plain)(case["op"], case, state)


def _framework(op, case, s):
    from precision_block_scaled_amd import pipeline as PL
    if op == "norm":
        amax = torch.empty(1, device=s["x"].device) if case["amax"] else None
        y, mean, rstd = PL.layernorm(s["x"], s["gamma"], s["beta"], EPS, out_dtype=TYPES[case["y"]], amax=amax)
        return dict(y=y, mean=mean, rstd=rstd, amax=None if amax is None else amax.to(y.dtype))
    if op == "norm_grad":
        dx, dgamma, dbeta = PL.layernorm_grad(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"])
        return dict(dx=dx, dgamma=dgamma, dbeta=dbeta)
    if op.startswith("xent"):
        loss, lse = PL.linear_xent(s["x"], s["w"], s["targets"])
        if op == "xent":
            return dict(loss=loss, lse=lse)
        dx, dw = PL.linear_xent_grad(s["dloss"], s["x"], s["w"], s["targets"], lse)
        return dict(loss=loss, lse=lse, dx=dx, dw=dw)
    loss, lse = PL.linear_distill(s["x"], s["w"], s["top_ids"], s["top_logits"], case["tau"])
    if op == "distill":
        return dict(loss=loss, lse=lse)
    dx, dw = PL.linear_distill_grad(s["dloss"], s["x"], s["w"], s["top_ids"], s["top_logits"], case["tau"], lse)
    return dict(loss=loss, lse=lse, dx=dx, dw=dw)


def _plain(op, case, s):
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1 / (d.square().mean(1) + EPS).sqrt()
        y = (d * rstd[:, None] * s["gamma"].float() + s["beta"].float()).to(TYPES[case["y"]])
        return dict(y=y, mean=mean, rstd=rstd, amax=y.abs().max().reshape(1) if case["amax"] else None)
    if op == "norm_grad":
        dy = s["dy"].float()
        n = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        u = dy * s["gamma"].float()
        dx = s["rstd"][:, None] * (u - u.mean(1, keepdim=True) - n * (u * n).mean(1, keepdim=True))
        return dict(dx=dx.to(s["x"].dtype), dgamma=(dy * n).sum(0), dbeta=dy.sum(0))

    x, w = s["x"].float(), s["w"].float()
    tau = case.get("tau", 1.0)
    z = x @ w.t() / tau
    high = z.max(1, keepdim=True).values
    e = (z - high).exp()
    total = e.sum(1, keepdim=True)
    lse = (high + total.log())[:, 0]
    if op.startswith("xent"):
        live = s["targets"] >= 0
        ids = s["targets"].clamp(min=0)[:, None]
        p = live.float()[:, None]
        own_entropy = 0.0
    else:
        held = s["top_ids"] >= 0
        live = held.any(1)
        ids = s["top_ids"].clamp(min=0)
        t = torch.where(held, s["top_logits"] / tau, -math.inf)
        t = t - torch.where(live, t.max(1).values, 0.0)[:, None]
        p = t.exp()
        sums = torch.where(live, p.sum(1), 1.0)[:, None]
        p = p / sums
        own_entropy = torch.where(p > 0, p * (t - sums.log()), 0.0).sum(1)
    loss = torch.where(live, own_entropy - (p * (z.gather(1, ids) - lse[:, None])).sum(1), 0.0)
    lse = torch.where(live, lse, 0.0)
    if not op.endswith("_grad"):
        return dict(loss=loss, lse=lse)
    scale = torch.where(live, s["dloss"], 0.0)[:, None] / tau
    dz = e.div_(total).scatter_add_(1, ids, -p).mul_(scale)
    return dict(loss=loss, lse=lse, dx=(dz @ w).bfloat16(), dw=(dz.t() @ x).bfloat16())


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    F = torch.nn.functional
    if op.startswith("norm"):
        x, gamma, beta = (s[k].double().requires_grad_() for k in ("x", "gamma", "beta"))
        y = F.layer_norm(x, (case["cols"],), gamma, beta, EPS)
        if op == "norm":
            var, mean = torch.var_mean(x.detach(), 1, correction=0)
            return dict(y=y.detach(), mean=mean, rstd=(var + EPS).rsqrt(),
                        amax=y.detach().abs().amax().reshape(1) if case["amax"] else None)
        dx, dgamma, dbeta = torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
        return dict(dx=dx, dgamma=dgamma, dbeta=dbeta)

    w = s["w"].double()
    grads = op.endswith("_grad")
    if grads:
        w.requires_grad_()
    tau = case.get("tau", 1.0)
    losses, lses, dxs, dw = [], [], [], torch.zeros_like(w) if grads else None
    for a in range(0, case["tokens"], 2048):
        rows = slice(a, a + 2048)
        x = s["x"][rows].double()
        if grads:
            x.requires_grad_()
        z = F.linear(x, w) / tau
        logq = F.log_softmax(z, 1)
        if op.startswith("xent"):
            live = s["targets"][rows] >= 0
            loss = F.nll_loss(logq, s["targets"][rows], ignore_index=IGNORE, reduction="none")
        else:
            held = s["top_ids"][rows] >= 0
            live = held.any(1)
            teacher = (s["top_logits"][rows].double() / tau).masked_fill(~held, -math.inf)
            logp = F.log_softmax(teacher.masked_fill(~live[:, None], 0.0), 1).masked_fill(~held, -math.inf)
            p = logp.exp()
            against = logq.gather(1, s["top_ids"][rows].clamp(min=0))
            loss = (torch.xlogy(p, p) - p * against).sum(1)
        losses.append(loss.detach())
        lses.append(torch.logsumexp(z.detach(), 1).masked_fill(~live, 0.0))
        if grads:
            dx, part = torch.autograd.grad((loss * s["dloss"][rows].double()).sum(), (x, w))
            dxs.append(dx)
            dw += part
    out = dict(loss=torch.cat(losses), lse=torch.cat(lses))
    if grads:
        out.update(dx=torch.cat(dxs), dw=dw)
    return out
