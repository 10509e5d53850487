"""The measured cases of the operators at a language model's ends: token
embedding, layer norm, and the output head's cross entropy, each with its
gradient.

`own` false computes them in plain form (elementary torch operations in fp32,
rounded once at the end); true makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
IGNORE = -100
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32, "int64": torch.int64}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # A short prompt's tokens in a small model: launch latency.
        dict(name="embed_prompt", op="embed", tokens=37, vocab=50257, dim=768, dtype="bf16", ids="int64"),
        # A training batch's tokens, most of them frequent ones.
        dict(name="embed_batch", op="embed", tokens=65536, vocab=131072, dim=4096, dtype="bf16", ids="int32"),
        # One sequence's gradient into the whole fp32 table of a small model.
        dict(name="embed_grad_sequence", op="embed_grad", tokens=1023, vocab=50257, dim=768, dtype="bf16", ids="int64"),
        # A training batch's gradient: repeated tokens, a few of them thousands of times.
        dict(name="embed_grad_batch", op="embed_grad", tokens=65536, vocab=131072, dim=2048, dtype="bf16", ids="int32"),
        # A few rows in fp32, odd length: launch latency.
        dict(name="norm_rows", op="norm", rows=17, dim=1001, dtype="fp32", weight="fp32"),
        # Every token of a training batch before one block.
        dict(name="norm_batch", op="norm", rows=65536, dim=4096, dtype="bf16", weight="fp32"),
        # One short sequence's gradient in a small model.
        dict(name="norm_grad_sequence", op="norm_grad", rows=517, dim=768, dtype="bf16", weight="bf16"),
        # A training batch's gradient in wide rows.
        dict(name="norm_grad_batch", op="norm_grad", rows=32768, dim=8192, dtype="bf16", weight="fp32"),
        # The loss alone, as an evaluation takes it: an odd vocabulary, an odd number of tokens.
        dict(name="head_eval", op="head", tokens=2047, vocab=50257, dim=1536, ignored=0.0, ids="int64"),
        # A handful of tokens: the table's reading and its gradient's writing are all of the work.
        dict(name="head_grad_few", op="head_grad", tokens=24, vocab=32000, dim=768, ignored=0.0, ids="int64"),
        # A fine-tuning step whose prompt tokens carry no loss.
        dict(name="head_grad_tuning", op="head_grad", tokens=1500, vocab=50257, dim=2048, ignored=0.5, ids="int64"),
        # A pre-training step over a large vocabulary.
        dict(name="head_grad_batch", op="head_grad", tokens=8192, vocab=131072, dim=2048, ignored=0.02, ids="int64"),
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of step."""
    n = max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)
    return n + step if n == 3072 else min(n, hi)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "head", "head_grad"])
    if op in ("embed", "embed_grad"):
        dim = rng.choice([_spread(rng, 64, 4096, 8), _spread(rng, 64, 4096)])
        vocab = _spread(rng, 1000, min(131072, 131072 * 2048 // dim))
        tokens = _spread(rng, 1, min(65536, 65536 * (4096 if op == "embed" else 2048) // dim // 2))
        return dict(op=op, tokens=tokens, vocab=vocab, dim=dim, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    ids=rng.choice(["int32", "int64"]))
    if op in ("norm", "norm_grad"):
        dim = rng.choice([_spread(rng, 64, 16384, 8), _spread(rng, 64, 16384)])
        rows = _spread(rng, 1, min(65536, 65536 * 4096 // dim // 2))
        return dict(op=op, rows=rows, dim=dim, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    weight=rng.choice(["fp32", "bf16"]))
    dim = _spread(rng, 64, 4096, 8)
    vocab = _spread(rng, 1000, 131072)
    tokens = _spread(rng, 1, max(2, min(8192, 8192 * 131072 * 1024 // (dim * vocab))))
    return dict(op=op, tokens=tokens, vocab=vocab, dim=dim, ignored=round(rng.choice([0.0, rng.uniform(0, 0.9)]), 2),
                ids=rng.choice(["int32", "int64"]))


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _randn(g, shape, scale, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _tokens(g, n, vocab, dtype):
    """Token ids in which low ids are frequent: id = floor(vocab u^4), so that
    id 0 is vocab^(-1/4) of all tokens."""
    u = torch.rand((n,), generator=g, device=DEV, dtype=torch.float64)
    return (u ** 4 * vocab).long().clamp_(0, vocab - 1).to(dtype)


def _distinct(n, vocab):
    """Expected number of distinct ids among n tokens drawn as in _tokens."""
    edge = (np.arange(vocab + 1) / vocab) ** 0.25
    p = np.minimum(np.diff(edge), 1.0 - 1e-16)
    return float(-np.expm1(n * np.log1p(-p)).sum())


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op in ("embed", "embed_grad"):
        t = TYPES[case["dtype"]]
        s["tok"] = _tokens(g, case["tokens"], case["vocab"], TYPES[case["ids"]])
        s["scale"] = math.sqrt(case["dim"])
        if op == "embed":
            s["table"] = _randn(g, (case["vocab"], case["dim"]), 0.02, t)
        else:
            s["dy"] = _randn(g, (case["tokens"], case["dim"]), 1e-3, t)
    elif op in ("norm", "norm_grad"):
        t, n, d = TYPES[case["dtype"]], case["rows"], case["dim"]
        s["w"] = _randn(g, (d,), 0.1, torch.float32).add_(1.0).to(TYPES[case["weight"]])
        s["b"] = _randn(g, (d,), 0.1, TYPES[case["weight"]])
        s["x"] = _randn(g, (n, d), 1.5, t).add_(0.25)
        if op == "norm_grad":
            # What the forward pass keeps for the backward pass.
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = (x - s["mean"][:, None]).square_().mean(1).add_(EPS).rsqrt_()
            s["dy"] = _randn(g, (n, d), 1e-3, t)
    else:
        n, v, d = case["tokens"], case["vocab"], case["dim"]
        s["h"] = _randn(g, (n, d), 1.0, torch.bfloat16)
        s["table"] = _randn(g, (v, d), 2.0 / math.sqrt(d), torch.bfloat16)
        tok = _tokens(g, n, v, torch.int64)
        drop = torch.rand((n,), generator=g, device=DEV) < case["ignored"]
        s["tok"] = torch.where(drop, torch.full_like(tok, IGNORE), tok).to(TYPES[case["ids"]])
    return s


# -------------------------------------------------------------------- runs --

def _plain(s):
    op = s["op"]
    if op == "embed":
        return (s["table"][s["tok"].long()].float() * s["scale"]).to(s["table"].dtype)
    if op == "embed_grad":
        out = torch.zeros((s["vocab"], s["dim"]), dtype=torch.float32, device=DEV)
        return out.index_add_(0, s["tok"].long(), s["dy"].float()).mul_(s["scale"])
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1.0 / ((c * c).mean(1) + EPS).sqrt()
        y = c * rstd[:, None] * s["w"].float() + s["b"].float()
        return y.to(s["x"].dtype), mean, rstd
    if op == "norm_grad":
        dy, w = s["dy"].float(), s["w"].float()
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        a = dy * w
        dx = (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
        return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    h, w, tok = s["h"].float(), s["table"].float(), s["tok"].long()
    live = (tok >= 0) & (tok < s["vocab"])
    at = torch.where(live, tok, torch.zeros_like(tok))[:, None]
    z = h @ w.t()
    top = z.amax(1, keepdim=True)
    zt = z.gather(1, at)
    p = (z - top).exp_()
    total = p.sum(1, keepdim=True)
    loss = torch.where(live, (total.log() + top - zt)[:, 0], torch.zeros_like(top[:, 0]))
    if op == "head":
        return loss
    g = live.float() / live.float().sum().clamp(min=1.0)
    p.mul_((g[:, None] / total)).scatter_add_(1, at, -g[:, None])
    return loss, (p @ w).to(torch.bfloat16), (p.t() @ h).to(torch.bfloat16)


def _own(s):
    import newton_schulz_07_gb300 as lib

    op = s["op"]
    if op == "embed":
        return lib.muon_embed(s["table"], s["tok"], scale=s["scale"])
    if op == "embed_grad":
        return lib.muon_embed_grad(s["dy"], s["tok"], s["vocab"], scale=s["scale"])
    if op == "norm":
        return lib.muon_layer_norm(s["x"], s["w"], s["b"], eps=EPS)
    if op == "norm_grad":
        return lib.muon_layer_norm_grad(s["dy"], s["x"], s["w"], s["mean"], s["rstd"])
    if op == "head":
        return lib.muon_head_loss(s["h"], s["table"], s["tok"], ignore_index=IGNORE)
    return lib.muon_head_loss_grad(s["h"], s["table"], s["tok"], ignore_index=IGNORE)


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4, "int32": 4, "int64": 8}
    if op in ("embed", "embed_grad"):
        t, v, d, e = case["tokens"], case["vocab"], case["dim"], size[case["dtype"]]
        ids = t * size[case["ids"]]
        if op == "embed":
            return {"bytes": ids + (_distinct(t, v) + t) * d * e, "flops": t * d}
        return {"bytes": ids + t * d * e + v * d * 4, "flops": t * d}
    if op in ("norm", "norm_grad"):
        n, d, e, w = case["rows"], case["dim"], size[case["dtype"]], size[case["weight"]]
        if op == "norm":
            return {"bytes": 2 * n * d * e + 2 * d * w + 8 * n, "flops": 8 * n * d}
        return {"bytes": 3 * n * d * e + d * (w + 8) + 8 * n, "flops": 14 * n * d}
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    read = 2 * d * (n + v) + n * size[case["ids"]] + 4 * n
    if op == "head":
        return {"bytes": read, "flops": 2 * n * v * d}
    return {"bytes": read + 2 * d * (n + v), "flops": 6 * n * v * d}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "embed":
        return torch.index_select(s["table"], 0, s["tok"].long()).to(f64) * s["scale"]
    if op == "embed_grad":
        order = torch.argsort(s["tok"].long(), stable=True)
        rows, count = torch.unique_consecutive(s["tok"].long()[order], return_counts=True)
        sums = torch.zeros((s["vocab"], s["dim"]), dtype=f64, device=DEV)
        last = torch.cumsum(count, 0)
        for c0 in range(0, s["dim"], 256):  # running sums of one slice of columns at a time
            run_ = torch.cumsum(s["dy"][order, c0:c0 + 256].to(f64), 0)
            upto = run_[last - 1]
            sums[rows, c0:c0 + 256] = torch.diff(upto, dim=0, prepend=torch.zeros_like(upto[:1])) * s["scale"]
        return sums
    if op == "norm":
        x = s["x"].to(f64)
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
        rstd = torch.pow(var + EPS, -0.5)
        return torch.addcmul(s["b"].to(f64), (x - mean[:, None]) * s["w"].to(f64), rstd[:, None]), mean, rstd
    if op == "norm_grad":
        d = case["dim"]
        dw = torch.zeros((d,), dtype=f64, device=DEV)
        db = torch.zeros_like(dw)
        dx = torch.empty(s["x"].shape, dtype=f64, device=DEV)
        for r in range(0, case["rows"], 4096):
            q = slice(r, r + 4096)
            rs = s["rstd"][q].to(f64)[:, None]
            xh, dy = (s["x"][q].to(f64) - s["mean"][q].to(f64)[:, None]) * rs, s["dy"][q].to(f64)
            dw += torch.einsum("nd,nd->d", dy, xh)
            db += torch.einsum("nd->d", dy)
            wy = torch.einsum("nd,d->nd", dy, s["w"].to(f64))
            dx[q] = rs * (wy - (wy.sum(1, keepdim=True) + xh * torch.einsum("nd,nd->n", wy, xh)[:, None]) / d)
        return dx, dw, db
    h, w, tok = s["h"].to(f64), s["table"].to(f64), s["tok"].long()
    ok = (tok != IGNORE).nonzero()[:, 0]
    loss = torch.zeros((case["tokens"],), dtype=f64, device=DEV)
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for r in range(0, ok.numel(), 2048):  # the rows that carry a loss, some at a time
        i = ok[r:r + 2048]
        z = torch.matmul(h[i], w.T)
        lse = torch.logsumexp(z, 1)
        here = torch.arange(i.numel(), device=DEV)
        loss[i] = lse - z[here, tok[i]]
        if op == "head_grad":
            dz = torch.exp(z - lse[:, None])
            dz[here, tok[i]] -= 1.0
            dz /= ok.numel()
            dh[i] = torch.matmul(dz, w)
            dw.addmm_(dz.T, h[i])
    return loss if op == "head" else (loss, dh, dw)
