"""Operators of a mixture-of-experts block in 8-bit floating point: what is measured, and its plain forms.

A block takes the residual stream's rows, normalises and quantises them, picks each token's
experts, runs the picked experts' two products on 8-bit codes, and adds the combined rows back to
the stream. Its operators, as this file names them in a case's "op":

  route    scores (sigmoid or softmax) of the router's logits, an optional balance bias for the
           choice, groups of experts of which the best are kept, top-k, renormalised weights
  quant    BF16 rows to E4M3 codes with one FP32 scale per row and 128 columns; with "swiglu" the
           rows are silu(gate) * up of a [gate | up] pair of halves
  product  E4M3 rows [M, K] (a scale per row and 128 of K) times E4M3 weights [N, K]^T (a scale per
           128 x 128 block), BF16 or FP32 out
  experts  the same product for every (token, slot) pair with its own expert's weights, the pairs
           grouped by expert in lists
  norm     the norm after a block, its gate and the residual's scale, and the norm before the next
           block: h = r + alpha * gate * rms(y), n = rms(h), with n's codes where asked; h goes
           on to n, and n to its codes, as they are before their own rounding

`run` computes the plain form (elementary torch operations in 32 bits, one rounding at the end)
unless `own` is set, when it makes the framework's calls.
"""
import math

import torch

own = False

BLOCK = 128  # columns (and weight rows) that share one scale
E4M3_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decoded token through the router of 896 experts: the softmax form, no groups; latency alone
        dict(name="route 1 x 896 softmax", op="route", tokens=1, experts=896, topk=16, scoring="softmax", bias=False, groups=1, kept=1, rule="max"),
        # a prompt of 4096 tokens, 256 experts in 8 groups of which 4 are kept by their two best, with the balance bias
        dict(name="route 4096 x 256 groups", op="route", tokens=4096, experts=256, topk=8, scoring="sigmoid", bias=True, groups=8, kept=4, rule="top2"),
        # one decoded hidden row on its way into an 8-bit product
        dict(name="quant 1 x 7168", op="quant", rows=1, cols=7168, swiglu=False, power=False),
        # the expert rows between the two products of a wide decode batch: 1020 tokens, 16 slots each
        dict(name="swiglu 16320 x 1024", op="quant", rows=16320, cols=1024, swiglu=True, power=False),
        # one decoded token's latent row up to the hidden size: the weights are read for one row
        dict(name="product 1", op="product", m=1, n=7168, k=3584, out="bf16"),
        # a ragged batch with FP32 output; n and k leave partial blocks of 96 rows and 16 columns
        dict(name="product 333 ragged", op="product", m=333, n=2016, k=7184, out="f32"),
        # a prompt's latent rows up to the hidden size
        dict(name="product 4096", op="product", m=4096, n=7168, k=3584, out="bf16"),
        # decode of 8 tokens, 16 of 896 experts each: about one row per picked expert, gate and up product
        dict(name="experts 8 of 896", op="experts", tokens=8, experts=896, topk=16, n=2048, k=3584, rows_in="token", out="bf16"),
        # the wide decode batch (204 requests x 5 tokens), about 18 rows per expert, down product
        dict(name="experts 1020 of 896", op="experts", tokens=1020, experts=896, topk=16, n=3584, k=1024, rows_in="pair", out="bf16"),
        # a prompt of 4096 tokens over 64 experts, 512 rows each: bound by the tensor cores
        dict(name="experts 4096 of 64", op="experts", tokens=4096, experts=64, topk=8, n=4096, k=3584, rows_in="token", out="bf16"),
        # one decoded token between two blocks, its codes for the next product made on the way
        dict(name="norm 1 x 7168", op="norm", tokens=1, hidden=7168, residual="bf16", gate="none", post=True, codes=True),
        # a prompt between two blocks: a gate for every value, the residual stream held in FP32
        dict(name="norm 4096 x 7168", op="norm", tokens=4096, hidden=7168, residual="f32", gate="full", post=True, codes=True),
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number between lo and hi, spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, min(hi // step * step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "quant", "product", "experts", "norm"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8, 16])
        size = rng.randint(8, 64) if groups > 1 else rng.randint(24, 1000)
        experts = groups * size
        kept = 1 if groups == 1 else rng.randint(1, groups)
        topk = rng.randint(1, min(16, kept * size))
        return dict(op=op, tokens=_spread(rng, 1, 4096), experts=experts, topk=topk, scoring=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.5,
                    groups=groups, kept=kept, rule=rng.choice(["top2", "max"]))
    if op == "quant":
        swiglu = rng.random() < 0.5
        return dict(op=op, rows=_spread(rng, 1, 16384), cols=_spread(rng, 128, 3584 if swiglu else 7168, 8), swiglu=swiglu, power=rng.random() < 0.5)
    if op == "product":
        return dict(op=op, m=_spread(rng, 1, 4096), n=_spread(rng, 64, 7168), k=_spread(rng, 128, 7168, 16), out=rng.choice(["bf16", "f32"]))
    if op == "experts":
        experts = rng.choice([16, 60, 64, 160, 256, 384])
        topk = rng.randint(1, 16)
        return dict(op=op, tokens=_spread(rng, 1, 2048), experts=experts, topk=topk, n=_spread(rng, 256, 4096, 8), k=_spread(rng, 256, 3584, 16),
                    rows_in=rng.choice(["token", "pair", "list"]), out=rng.choice(["bf16", "f32"]))
    return dict(op=op, tokens=_spread(rng, 1, 4096), hidden=_spread(rng, 128, 7168, 8), residual=rng.choice(["bf16", "f32"]),
                gate=rng.choice(["none", "token", "channel", "full"]), post=rng.random() < 0.75, codes=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------
# inputs

def _blocks(n):
    return -(-n // BLOCK)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _padded(x, cols):
    """x with its last dimension padded with zeros to `cols`."""
    return x if x.shape[-1] == cols else torch.nn.functional.pad(x, (0, cols - x.shape[-1]))


def _code_rows(g, rows, k):
    """Activations on their codes: rows ~ N(0, 1) with a few large channels, quantised by 128."""
    nb = _blocks(k)
    x = _normal(g, rows, k) * (1.0 + 9.0 * (torch.rand(k, generator=g, device="cuda") < 0.01))
    b = _padded(x, nb * BLOCK).view(rows, nb, BLOCK)
    amax = b.abs().amax(-1).clamp_min(1e-6)
    codes = (b * (E4M3_MAX / amax)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, nb * BLOCK)[:, :k]
    return codes.contiguous().to(torch.float8_e4m3fn).view(torch.uint8), amax / E4M3_MAX


def _code_weights(g, *shape):
    """Weights on their codes, about N(0, 0.02): the codes ~ N(0, 100), a scale per 128 x 128 block."""
    n, k = shape[-2:]
    q = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = q.view(-1)
    step = 1 << 28
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        part.copy_(_normal(g, part.numel()).mul_(100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
    s = (0.02 / 100.0) * torch.exp(0.3 * _normal(g, *shape[:-2], _blocks(n), _blocks(k)))
    return q, s


def _near(case, logits, bias):
    """The tokens whose choice hangs on the last bits of a score: two keys in 64 bits that differ,
    by less than any 32-bit evaluation is sure to tell apart."""
    x = logits.double()
    s = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, -1)
    key = s if bias is None else s + bias.double()
    t, groups, kept = case["tokens"], case["groups"], case["kept"]

    def close(v):
        d = v[:, :-1] - v[:, 1:]
        return (d > 0) & (d < 4e-6 * v[:, :-1].abs().clamp_min(1e-3 if bias is not None else 1e-12))

    bad = torch.zeros(t, dtype=torch.bool, device=x.device)
    if groups > 1:
        by = key.view(t, groups, -1)
        score = by.amax(-1) if case["rule"] == "max" else by.topk(min(2, by.shape[-1]), -1).values.sum(-1)
        top = torch.sort(score, dim=-1, descending=True, stable=True)
        if kept < groups:
            bad |= close(top.values[:, kept - 1:kept + 1]).any(-1)
        keep = torch.zeros(t, groups, dtype=torch.bool, device=x.device).scatter_(1, top.indices[:, :kept], True)
        key = by.masked_fill(~keep[..., None], -math.inf).view(t, -1)
    order = torch.sort(key, -1, descending=True).values[:, :case["topk"] + 1]
    return bad | close(order).any(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    dev = dict(device="cuda")
    s = dict(case=dict(case))
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        logits = _normal(g, t, e).to(torch.bfloat16).float()  # a router that computes in BF16: equal logits do occur
        bias = (_normal(g, e) * 0.05).to(torch.bfloat16).float() if case["bias"] else None
        # A token whose order hangs on the last bits of a score has no answer that two right programs share: drawn again.
        while (at := _near(case, logits, bias).nonzero()[:, 0]).numel():
            logits[at] = _normal(g, at.numel(), e).to(torch.bfloat16).float()
        s.update(logits=logits, bias=bias, ids=torch.empty(t, k, dtype=torch.int32, **dev), weights=torch.empty(t, k, **dev),
                 weights_bf16=torch.empty(t, k, dtype=torch.bfloat16, **dev))
    elif op == "quant":
        rows, cols = case["rows"], case["cols"]
        width = 2 * cols if case["swiglu"] else cols
        x = _normal(g, rows, width) * torch.exp(0.5 * _normal(g, rows, 1))
        s.update(x=x.to(torch.bfloat16), q=torch.empty(rows, cols, dtype=torch.uint8, **dev), scales=torch.empty(rows, _blocks(cols), **dev))
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a, sa = _code_rows(g, m, k)
        w, sw = _code_weights(g, n, k)
        s.update(a=a, sa=sa, w=w, sw=sw, out=torch.empty(m, n, dtype=_dtype(case["out"]), **dev))
    elif op == "experts":
        t, e, topk, n, k = (case[v] for v in ("tokens", "experts", "topk", "n", "k"))
        ids = (_normal(g, t, e) + 0.3 * _normal(g, e)).topk(topk, -1).indices  # some experts are asked for more often
        pairs = torch.sort(ids.reshape(-1), stable=True).indices.to(torch.int32)
        counts = torch.bincount(ids.reshape(-1), minlength=e)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        a, sa = _code_rows(g, t if case["rows_in"] == "token" else t * topk, k)
        w, sw = _code_weights(g, e, n, k)
        s.update(a=a, sa=sa, w=w, sw=sw, offsets=offsets, pairs=pairs, out=torch.empty(t * topk, n, dtype=_dtype(case["out"]), **dev))
    else:
        t, h = case["tokens"], case["hidden"]
        gate = {"none": None, "token": (t, 1), "channel": (h,), "full": (t, h)}[case["gate"]]
        s.update(y=_normal(g, t, h).mul_(3.0).to(torch.bfloat16), residual=_normal(g, t, h).mul_(2.0).to(_dtype(case["residual"])),
                 post=(1.0 + 0.1 * _normal(g, h)).to(torch.bfloat16) if case["post"] else None,
                 next=(1.0 + 0.1 * _normal(g, h)).to(torch.bfloat16),
                 gate=None if gate is None else (1.0 + 0.5 * _normal(g, *gate)).to(torch.bfloat16),
                 h=torch.empty(t, h, dtype=_dtype(case["residual"]), **dev), n=torch.empty(t, h, dtype=torch.bfloat16, **dev),
                 q=torch.empty(t, h, dtype=torch.uint8, **dev) if case["codes"] else None,
                 scales=torch.empty(t, _blocks(h), **dev) if case["codes"] else None)
    return s


ROUTE_SCALE = 2.5  # the routed experts' factor
ALPHA = 0.7        # the residual scale of a block


# ---------------------------------------------------------------------------------------------
# one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _e4m3(q):
    return q.view(torch.float8_e4m3fn)


def _run_own(s):
    import latent_moe_decode_gb300 as m

    c = s["case"]
    op = c["op"]
    if op == "route":
        return m.topk_route_grouped(
            s["logits"], s["bias"], c["topk"], n_group=c["groups"], topk_group=c["kept"],
            scoring=m.SCORE_SIGMOID if c["scoring"] == "sigmoid" else m.SCORE_SOFTMAX,
            group_rule=m.GROUP_TOP2 if c["rule"] == "top2" else m.GROUP_MAX, renormalize=True, scale=ROUTE_SCALE,
            ids=s["ids"], weights=s["weights"], weights_bf16=s["weights_bf16"])
    if op == "quant":
        call = m.fp8_block_quantize_swiglu if c["swiglu"] else m.fp8_block_quantize_rows
        q, scales = call(s["x"], q=s["q"], scales=s["scales"], scale_rule=m.FP8_SCALE_POW2 if c["power"] else m.FP8_SCALE_AMAX)
        return _e4m3(q), scales
    if op == "product":
        return m.fp8_block_gemm(s["a"], s["sa"], s["w"], s["sw"], out=s["out"])
    if op == "experts":
        rows = {"token": m.ROWS_TOKEN, "pair": m.ROWS_PAIR, "list": m.ROWS_LIST}
        return m.expert_gemm(s["a"], s["sa"], s["w"], s["sw"], s["offsets"], s["pairs"], c["topk"], in_rows=rows[c["rows_in"]],
                             out_rows=m.ROWS_PAIR, out=s["out"])
    h, n, q, scales = m.block_norm(s["y"], s["residual"], s["next"], post_weight=s["post"], gate=s["gate"], alpha=ALPHA, eps=EPS,
                                   h=s["h"], n=s["n"], quantize=c["codes"], q=s["q"], scales=s["scales"])
    return (h, n, _e4m3(q), scales) if c["codes"] else (h, n)


def _codes(x, power=False):
    """(E4M3 codes, scales) of FP32 rows, a scale for each 128 columns: amax / 448, or the power of
    two at or above it."""
    rows, cols = x.shape
    nb = _blocks(cols)
    b = _padded(x, nb * BLOCK).view(rows, nb, BLOCK)
    amax = b.abs().amax(-1)
    if power:
        mant, ex = torch.frexp(amax / E4M3_MAX)
        ex = torch.where(mant == 0.5, ex - 1, ex).clamp(-126, 127)
        scale, mult = ((ex + 127) << 23).view(torch.float32), ((127 - ex) << 23).view(torch.float32)  # 2^ex, 2^-ex
    else:
        scale = amax / E4M3_MAX
        mult = E4M3_MAX / amax
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    mult = torch.where(amax == 0, torch.ones_like(mult), mult)
    q = (b * mult[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, nb * BLOCK)[:, :cols]
    return q.contiguous().to(torch.float8_e4m3fn), scale


def _real_rows(q, scales):
    """FP32 values of code rows [M, K] with a scale per row and 128 columns."""
    return _e4m3(q).float() * scales.repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _real_weights(w, scales):
    """FP32 values of code weights [..., N, K] with a scale per 128 x 128 block."""
    n, k = w.shape[-2:]
    v = _e4m3(w).float()
    return v.mul_(scales.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k])


def _rms(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        x, t = s["logits"], c["tokens"]
        if c["scoring"] == "sigmoid":
            score = 1.0 / (1.0 + torch.exp(-x))
        else:
            e = torch.exp(x - x.amax(-1, keepdim=True))
            score = e / e.sum(-1, keepdim=True)
        key = score if s["bias"] is None else score + s["bias"]
        if c["groups"] > 1:
            by = key.view(t, c["groups"], -1)
            if c["rule"] == "max":
                best = by.amax(-1)
            else:
                best = torch.sort(by, -1, descending=True).values[..., :2].sum(-1)
            kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, : c["kept"]]
            mask = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
            key = by.masked_fill(~mask[..., None], -math.inf).view(t, -1)
        ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, : c["topk"]]
        w = score.gather(1, ids)
        w = w / w.sum(-1, keepdim=True) * ROUTE_SCALE
        return ids.to(torch.int32), w, w.to(torch.bfloat16)
    if op == "quant":
        x = s["x"].float()
        if c["swiglu"]:
            gate, up = x.chunk(2, -1)
            x = gate / (1.0 + torch.exp(-gate)) * up
        return _codes(x, c["power"])
    if op == "product":
        return (_real_rows(s["a"], s["sa"]) @ _real_weights(s["w"], s["sw"]).t()).to(_dtype(c["out"]))
    if op == "experts":
        pairs, offsets = s["pairs"].long(), s["offsets"].long()
        counts = offsets[1:] - offsets[:-1]
        active = counts.nonzero()[:, 0]  # the experts with rows, and the rows of the fullest: read on the host
        cap = int(counts.max())
        at = torch.repeat_interleave(torch.arange(active.numel(), device=pairs.device), counts[active], output_size=pairs.numel())
        place = torch.arange(pairs.numel(), device=pairs.device) - offsets[active][at]
        row = {"token": pairs // c["topk"], "pair": pairs, "list": torch.arange(pairs.numel(), device=pairs.device)}[c["rows_in"]]
        a = torch.zeros(active.numel(), cap, c["k"], device=pairs.device)
        a[at, place] = _real_rows(s["a"], s["sa"])[row]
        v = torch.bmm(a, _real_weights(s["w"][active], s["sw"][active]).transpose(1, 2))
        out = torch.empty(pairs.numel(), c["n"], dtype=_dtype(c["out"]), device=pairs.device)
        out[pairs] = v[at, place].to(out.dtype)
        return out
    y = s["y"].float()
    if s["post"] is not None:
        y = _rms(y, s["post"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = s["residual"].float() + ALPHA * y
    n = _rms(h, s["next"])
    out = h.to(s["residual"].dtype), n.to(torch.bfloat16)
    return (*out, *_codes(n)) if c["codes"] else out


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits

def _exact_scales(x, power=False):
    nb = _blocks(x.shape[1])
    amax = torch.stack([x[:, i * BLOCK:(i + 1) * BLOCK].abs().amax(1) for i in range(nb)], 1)
    scale = amax / E4M3_MAX
    if power:  # the smallest power of two with amax <= 448 * scale
        scale = ((torch.floor(torch.log2(scale)).clamp(-1000).long() + 1022) << 52).view(torch.float64)  # half of it or less
        for _ in range(3):
            scale = torch.where(amax > E4M3_MAX * scale, 2 * scale, scale)
    return torch.where(amax == 0, torch.ones_like(scale), scale)


def _exact_codes(x, power=False):
    """x / scale on the grid of E4M3 (three bits after the leading one, steps of 2^-9 below 2^-6),
    ties to the even step."""
    scale = _exact_scales(x, power)
    v = x / scale[:, torch.arange(x.shape[1], device=x.device) // BLOCK]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x = s["logits"].double()
        p = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, 1)
        key = p.clone() if s["bias"] is None else p + s["bias"].double()
        if case["groups"] > 1:
            size = case["experts"] // case["groups"]
            per = key.reshape(case["tokens"], case["groups"], size).sort(-1, descending=True).values
            value = per[..., 0] if case["rule"] == "max" or size == 1 else per[..., 0] + per[..., 1]
            rank = value.argsort(dim=1, descending=True, stable=True).argsort(dim=1)
            key[(rank >= case["kept"]).repeat_interleave(size, 1)] = -math.inf
        ids = key.argsort(dim=1, descending=True, stable=True)[:, : case["topk"]]
        w = torch.gather(p, 1, ids)
        w = ROUTE_SCALE * w / w.sum(1, keepdim=True)
        return ids.to(torch.int32), w, w
    if op == "quant":
        x = s["x"].double()
        if case["swiglu"]:
            f = case["cols"]
            x = x[:, :f] * torch.sigmoid(x[:, :f]) * x[:, f:]
        return _exact_codes(x, case["power"])
    if op in ("product", "experts"):
        def real(q, scale, rows_per_scale):
            n, k = q.shape
            v = q.view(torch.float8_e4m3fn).double()
            i = torch.arange(n, device=q.device)[:, None] // rows_per_scale
            return v * scale.double()[i, torch.arange(k, device=q.device)[None] // BLOCK]

        a = real(s["a"], s["sa"], 1)
        if op == "product":
            return a @ real(s["w"], s["sw"], BLOCK).t()
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        ends, pairs = s["offsets"].tolist(), s["pairs"].long()
        for e in range(case["experts"]):
            lo, hi = ends[e], ends[e + 1]
            if lo < hi:
                p = pairs[lo:hi]
                rows = {"token": p // case["topk"], "pair": p, "list": torch.arange(lo, hi, device=p.device)}[case["rows_in"]]
                out[p] = a[rows] @ real(s["w"][e], s["sw"][e], BLOCK).t()
        return out
    y = s["y"].double()
    if s["post"] is not None:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * s["post"].double()
    if s["gate"] is not None:
        y = s["gate"].double() * y
    h = s["residual"].double() + ALPHA * y
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["next"].double()
    return (h, n, *_exact_codes(n)) if case["codes"] else (h, n)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        return {"bytes": 4 * t * e + (4 * e if case["bias"] else 0) + 10 * t * k, "flops": 8 * t * e}
    if op == "quant":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": rows * ((4 if case["swiglu"] else 2) * cols + cols + 4 * _blocks(cols)), "flops": (8 if case["swiglu"] else 3) * rows * cols}
    size = 4 if case.get("out") == "f32" else 2
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * (k + 4 * _blocks(k)) + n * k + 4 * _blocks(n) * _blocks(k) + size * m * n, "flops": 2 * m * n * k}
    if op == "experts":
        t, e, topk, n, k = (case[v] for v in ("tokens", "experts", "topk", "n", "k"))
        active = e * (1.0 - (1.0 - topk / e) ** t)  # experts that some token picked
        rows = t if case["rows_in"] == "token" else t * topk
        return {"bytes": int(active * (n * k + 4 * _blocks(n) * _blocks(k)) + rows * (k + 4 * _blocks(k)) + t * topk * (size * n + 4) + 4 * e),
                "flops": 2 * t * topk * n * k}
    t, h = case["tokens"], case["hidden"]
    r = 4 if case["residual"] == "f32" else 2
    gate = {"none": 0, "token": 2 * t, "channel": 2 * h, "full": 2 * t * h}[case["gate"]]
    codes = t * (h + 4 * _blocks(h)) if case["codes"] else 0
    return {"bytes": t * h * (2 + 2 * r + 2) + gate + (4 if case["post"] else 2) * h + codes, "flops": 12 * t * h}
