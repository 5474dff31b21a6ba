"""What is measured of the operators on either side of the head: the norm of the residual stream before
it, the clipping of the gradients after it, and the penalties, biases and masks on its logits.

``run`` computes each in elementary torch operations, or, where ``own`` is true, by the calls that a
user of the package makes.  ``exact`` is each operator's definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a decoding step through the final norm of a 4096-wide model: latency
        {"name": "norm-decode-1", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "res": "bf16", "offset": 0.0},
        # the final norm of a training step of 16384 tokens, forward
        {"name": "norm-train-fwd", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "res": "bf16",
         "offset": 0.0},
        # the same, backward: the head's gradient in, the residual stream's gradient and dweight out
        {"name": "norm-train-bwd", "op": "norm-bwd", "rows": 16384, "cols": 4096, "dtype": "bf16", "res": "bf16",
         "offset": 0.0},
        # a ragged batch with an odd width, an fp32 residual stream and the (1 + w) form, backward
        {"name": "norm-ragged-bwd", "op": "norm-bwd", "rows": 4099, "cols": 1283, "dtype": "bf16", "res": "f32",
         "offset": 1.0},
        # a prefill of 8192 tokens whose next product takes 8-bit operands: a scale for each 128 columns
        {"name": "norm-fp8-prefill", "op": "norm-fp8", "rows": 8192, "cols": 2048, "dtype": "f16", "res": "f16",
         "offset": 0.0, "group": 128},
        # the gradients of rank-16 adapters: many small tensors
        {"name": "clip-adapters", "op": "clip", "kind": "adapters", "tensors": 112, "rows": 16, "cols": 2048,
         "dtype": "bf16", "clipped": True},
        # the gradients of a 151936 x 4096 head with its bias and norm weight
        {"name": "clip-head", "op": "clip", "kind": "head", "tensors": 3, "rows": 151936, "cols": 4096, "dtype": "bf16",
         "clipped": True},
        # fp32 gradients of a small model's layers, of odd sizes, whose norm is below the limit
        {"name": "clip-odd-f32", "op": "clip", "kind": "odd", "tensors": 37, "rows": 1013, "cols": 1283, "dtype": "f32",
         "clipped": False},
        # one request's next token: 1000 tokens of history
        {"name": "logits-decode-1", "op": "logits", "rows": 1, "vocab": 151936, "dtype": "f32", "history": 1000,
         "biases": 8, "mask": True, "ids32": False},
        # a serving batch with bf16 logits, long histories, biases and grammar masks
        {"name": "logits-batch-64", "op": "logits", "rows": 64, "vocab": 128256, "dtype": "bf16", "history": 4096,
         "biases": 64, "mask": True, "ids32": False},
        # an odd batch and vocabulary with very long histories, no mask
        {"name": "logits-ragged-long", "op": "logits", "rows": 37, "vocab": 100003, "dtype": "f16", "history": 32768,
         "biases": 0, "mask": False, "ids32": True},
        # the largest batch: 256 requests over a 262144-word vocabulary
        {"name": "logits-batch-256", "op": "logits", "rows": 256, "vocab": 262144, "dtype": "f32", "history": 2048,
         "biases": 300, "mask": True, "ids32": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A size between lo and hi: a multiple of 128, of 8, or any."""
    n = _log_int(rng, lo, hi)
    step = rng.choice([128, 8, 8, 1])
    n = max(lo, n // step * step)
    return n if n != 3072 else n + 8


def draw(rng):
    op = rng.choice(["norm", "norm-bwd", "norm-fp8", "clip", "logits", "logits"])
    if op in ("norm", "norm-bwd", "norm-fp8"):
        cols = _width(rng, 128, 16384)
        rows = _log_int(rng, 1, min(16384, 16384 * 4096 // cols))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op == "norm-fp8" and dtype == "f32":
            dtype = "bf16"
        case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "res": rng.choice([dtype, dtype, "f32"]),
                "offset": rng.choice([0.0, 0.0, 1.0])}
        if op == "norm-fp8":
            case["group"] = rng.choice([0, 32, 64, 128])
        return case
    if op == "clip":
        kind = rng.choice(["adapters", "odd", "odd", "head"])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if kind == "adapters":
            tensors, rows, cols = rng.randint(2, 300), rng.choice([4, 8, 16, 64]), _width(rng, 128, 8192)
        elif kind == "odd":
            tensors, rows, cols = rng.randint(1, 60), _log_int(rng, 1, 1500), _width(rng, 128, 2048)
        else:
            tensors, rows, cols = 3, _width(rng, 1000, 150000), _width(rng, 128, 2048)
        return {"op": "clip", "kind": kind, "tensors": tensors, "rows": rows, "cols": cols, "dtype": dtype,
                "clipped": rng.random() < 0.75}
    vocab = _width(rng, 1000, 262144)
    rows = _log_int(rng, 1, 256)
    return {"op": "logits", "rows": rows, "vocab": vocab, "dtype": rng.choice(["f32", "bf16", "f16"]),
            "history": _log_int(rng, 1, 32768 if rows <= 64 else 4096), "biases": rng.choice([0, 0, 1, 32, 300]),
            "mask": rng.random() < 0.6, "ids32": rng.random() < 0.5}


def _clip_shapes(case):
    rows, cols = case["rows"], case["cols"]
    if case["kind"] == "adapters":  # A and B of each adapter
        return [(rows, cols) if i % 2 == 0 else (cols, rows) for i in range(case["tensors"])]
    if case["kind"] == "head":      # dweight, dbias, the norm's dweight
        return [(rows, cols), (rows,), (cols,)]
    return [(rows + 7 * i, cols - (i * 31) % 97) if i % 3 else (cols + i,) for i in range(case["tensors"])]


def _group(case):
    """Columns per scale; 0 stands for the whole row, and the last group of a row may be short."""
    return case["group"] or case["cols"]


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kw = dict(generator=g, device="cuda", dtype=torch.float32)
    st = {"case": case}
    if case["op"].startswith("norm"):
        n, d = case["rows"], case["cols"]
        t, r = DTYPES[case["dtype"]], DTYPES[case["res"]]
        w = torch.randn(d, **kw) * 0.2
        st["weight"] = (w if case["offset"] else w + 1.0).to(t)
        # the residual stream's columns differ in size, a few by far
        col = torch.exp(torch.randn(d, **kw))
        if case["op"] == "norm-bwd":
            h = (torch.randn(n, d, **kw) * 2.0 * col).to(r)
            st["h"] = h
            st["dy"] = (torch.randn(n, d, **kw) * 1e-2).to(t)
            st["dh"] = (torch.randn(n, d, **kw) * 1e-2).to(r)
            # what the forward of this training step kept
            st["rstd"] = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
        else:
            st["x"] = torch.randn(n, d, **kw).to(t)
            st["residual"] = (torch.randn(n, d, **kw) * 2.0 * col).to(r)
        return st
    if case["op"] == "clip":
        t = DTYPES[case["dtype"]]
        shapes = _clip_shapes(case)
        scale = 10.0 ** (-4.0 * torch.rand(len(shapes), generator=g, device="cuda"))
        st["grads"] = [(torch.randn(s, **kw) * scale[i]).to(t) for i, s in enumerate(shapes)]
        if len(shapes) > 3:
            st["grads"][2].zero_()  # a parameter that this batch did not touch
        # the optimizer's flat buffer takes the clipped gradients
        sizes = [x.numel() for x in st["grads"]]
        st["flat"] = torch.empty(sum(sizes), dtype=t, device="cuda")
        st["out"] = [f.view(s) for f, s in zip(st["flat"].split(sizes), shapes)]
        st["max_norm"] = 5e-5 * math.sqrt(sum(sizes)) if case["clipped"] else 10.0 * math.sqrt(sum(sizes))
        return st
    b, v, n = case["rows"], case["vocab"], case["history"]
    ids = torch.int32 if case["ids32"] else torch.int64
    z = torch.randn(b, v, **kw) * 3.0
    # texts repeat a few words often: ids crowd at the low end of a cube law
    st["tokens"] = (v * torch.rand(b, n, generator=g, device="cuda", dtype=torch.float64).pow(3)).long() \
        .clamp_(max=v - 1).to(ids)
    # histories of different lengths, prompts of a half on average; a first token has no output yet
    st["lens"] = (n * (0.25 + 0.75 * torch.rand(b, generator=g, device="cuda"))).long().clamp_(min=1, max=n)
    st["prompt_lens"] = (st["lens"] * torch.rand(b, generator=g, device="cuda")).long()
    st["repetition"] = 1.0 + 0.3 * torch.rand(b, **kw)
    st["presence"] = torch.rand(b, **kw) - 0.25
    st["frequency"] = 0.5 * torch.rand(b, **kw)
    z[:, v - 1 - v // 50:] = float("-inf")  # the padding of the vocabulary
    st["logits"] = z.to(DTYPES[case["dtype"]])
    st["bias_ids"] = st["bias"] = st["mask"] = None
    if case["biases"]:
        k = min(case["biases"], v)
        first = torch.randint(0, v, (b, 1), generator=g, device="cuda")
        st["bias_ids"] = ((first + 17 * torch.arange(k, device="cuda")) % v).to(ids)
        st["bias"] = torch.randn(b, k, **kw) * 5.0
    if case["mask"]:
        words = (v + 31) // 32
        m = torch.randint(-2 ** 31, 2 ** 31, (b, words), generator=g, device="cuda").to(torch.int32)
        row = torch.arange(b, device="cuda")[:, None]
        m = torch.where(row % 4 == 0, torch.full_like(m, -1), m)          # free text
        few = torch.zeros_like(m)
        few[:, : max(1, words // 500)] = 0x00F00F01
        m = torch.where(row % 4 == 3, few, m)                             # a few words allowed
        st["mask"] = torch.where(row % 32 == 31, torch.zeros_like(m), m)  # a grammar at its end: nothing
    return st


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------
def run(st):
    case = st["case"]
    if own:
        return _run_own(case, st)
    if case["op"] == "norm":
        return _plain_norm(case, st)
    if case["op"] == "norm-fp8":
        return _plain_norm_fp8(case, st)
    if case["op"] == "norm-bwd":
        return _plain_norm_bwd(case, st)
    if case["op"] == "clip":
        return _plain_clip(st)
    return _plain_logits(st)


def _run_own(case, st):
    import linear_cross_entropy_tmem_gb300 as flce
    if case["op"] == "norm":
        r = flce.flce_add_rms_norm(st["x"], st["weight"], st["residual"], eps=1e-6, weight_offset=case["offset"],
                                   need_rstd=False)
        return r.y, r.h
    if case["op"] == "norm-fp8":
        r = flce.flce_add_rms_norm_fp8(st["x"], st["weight"], st["residual"], eps=1e-6,
                                       weight_offset=case["offset"], group=case["group"])
        return r.q, r.scale, r.h
    if case["op"] == "norm-bwd":
        r = flce.flce_add_rms_norm_backward(st["dy"], st["h"], st["rstd"], st["weight"], dh=st["dh"],
                                            weight_offset=case["offset"])
        return r.dx, r.dresidual, r.dweight
    if case["op"] == "clip":
        norm = flce.clip_grad_norm_(st["grads"], st["max_norm"], outputs=st["out"])
        return norm, st["flat"]
    r = flce.process_logits(st["logits"], tokens=st["tokens"], lens=st["lens"], prompt_lens=st["prompt_lens"],
                            repetition=st["repetition"], presence=st["presence"], frequency=st["frequency"],
                            bias_ids=st["bias_ids"], bias=st["bias"], mask=st["mask"])
    return r.logits, r.token, r.lse


def _normed(case, st):
    h = (st["x"].float() + st["residual"].float()).to(st["residual"].dtype)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(1, keepdim=True) + 1e-6)
    return f * rstd * (st["weight"].float() + case["offset"]), h


def _plain_norm(case, st):
    y, h = _normed(case, st)
    return y.to(st["x"].dtype), h


def _plain_norm_fp8(case, st):
    y, h = _normed(case, st)
    n, d = y.shape
    size = _group(case)
    groups = -(-d // size)
    y = torch.nn.functional.pad(y, (0, groups * size - d)).view(n, groups, size)
    scale = y.abs().amax(2) / E4M3_MAX
    q = torch.where(scale[..., None] > 0, y / scale[..., None], torch.zeros_like(y))
    q = q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(n, groups * size)[:, :d], scale, h


def _plain_norm_bwd(case, st):
    dy, h, rstd = st["dy"].float(), st["h"].float(), st["rstd"][:, None]
    xh = h * rstd
    g = dy * (st["weight"].float() + case["offset"])
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True)) + st["dh"].float()
    return dx.to(st["dy"].dtype), dx.to(st["h"].dtype), (dy * xh).sum(0).to(st["weight"].dtype)


def _plain_clip(st):
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]])
    norm = squares.sum().sqrt().float()
    c = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
    _ = [o.copy_(g.float() * c) for o, g in zip(st["out"], st["grads"])]
    return norm, st["flat"]


def _plain_logits(st):
    z = st["logits"].float()
    b, v = z.shape
    t = st["tokens"].long()
    at = torch.arange(t.shape[1], device=t.device)[None]
    live = at < st["lens"][:, None]
    answered = live & (at >= st["prompt_lens"][:, None])
    seen = torch.zeros(b, v, dtype=torch.int32, device=t.device).scatter_add_(1, t, live.int()) > 0
    count = torch.zeros(b, v, dtype=torch.int32, device=t.device).scatter_add_(1, t, answered.int())
    rep = st["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - st["frequency"][:, None] * count.float()
    z = torch.where(count > 0, z - st["presence"][:, None], z)
    if st["bias"] is not None:
        z = z + torch.zeros_like(z).scatter_add_(1, st["bias_ids"].long(), st["bias"])
    if st["mask"] is not None:
        word = st["mask"].long()[:, :, None] >> torch.arange(32, device=t.device)
        z = torch.where((word & 1).view(b, -1)[:, :v] > 0, z, torch.full_like(z, float("-inf")))
    out = z.to(st["logits"].dtype)
    f = out.float()
    top = f.amax(1)
    token = torch.where(f == top[:, None], torch.arange(v, device=t.device)[None], v).amin(1)
    token = torch.where(top == float("-inf"), -1, token)
    base = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    lse = base + torch.exp(f - base[:, None]).sum(1).log()
    return out, token, lse


# ---------------------------------------------------------------------------------------------------
# Work, and the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------
def work(case):
    if case["op"].startswith("norm"):
        n, d = case["rows"], case["cols"]
        t, r = BYTES[case["dtype"]], BYTES[case["res"]]
        if case["op"] == "norm-bwd":
            # read dy, h, dh, rstd, w; write the gradient in each type that is asked for, and dw
            wrote = t if case["dtype"] == case["res"] else t + r
            return {"bytes": n * d * (t + 2 * r + wrote) + 4 * n + 2 * d * t, "flops": 12.0 * n * d}
        y = 1 if case["op"] == "norm-fp8" else t
        scales = 4 * n * -(-d // _group(case)) if case["op"] == "norm-fp8" else 0
        return {"bytes": n * d * (t + 2 * r + y) + scales + d * t, "flops": 8.0 * n * d}
    if case["op"] == "clip":
        n = sum(math.prod(s) for s in _clip_shapes(case))
        return {"bytes": 2 * n * BYTES[case["dtype"]] + 4, "flops": 3.0 * n}
    b, v = case["rows"], case["vocab"]
    ids = 4 if case["ids32"] else 8
    row = 2 * v * BYTES[case["dtype"]] + case["history"] * ids * 5 // 8 + case["biases"] * (ids + 4) + 40
    row += 4 * ((v + 31) // 32) if case["mask"] else 0
    return {"bytes": b * row, "flops": 6.0 * b * v}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("norm", "norm-fp8"):
        kept = st["residual"].dtype
        h = torch.add(st["x"].double(), st["residual"].double()).to(kept)
        y = h.double()
        y /= torch.sqrt(torch.mul(y, y).sum(-1) / case["cols"] + 1e-6).unsqueeze(-1)
        y *= st["weight"].double().add(case["offset"]).unsqueeze(0)
        if case["op"] == "norm":
            return y, h.double()
        parts = y.split(_group(case), dim=1)
        s = [p.abs().max(1).values / E4M3_MAX for p in parts]
        q = [(p / k.clamp(min=1e-300).unsqueeze(1)).float().to(torch.float8_e4m3fn).double() for p, k in zip(parts, s)]
        return torch.cat(q, 1), torch.stack(s, 1), h.double()
    if case["op"] == "norm-bwd":
        h, rho, dy = st["h"].double(), st["rstd"].double().unsqueeze(1), st["dy"].double()
        g = dy * st["weight"].double().add(case["offset"])
        dot = torch.einsum("nd,nd->n", g, h).unsqueeze(1)
        dx = g * rho - h * dot * rho.pow(3) / case["cols"] + st["dh"].double()
        return dx, dx, torch.einsum("nd,nd->d", dy, h * rho)
    if case["op"] == "clip":
        flat = torch.cat([g.reshape(-1) for g in st["grads"]]).double()
        norm = math.sqrt(float(torch.dot(flat, flat)))
        return torch.tensor(norm, dtype=torch.float64), flat.mul_(min(1.0, st["max_norm"] / (norm + 1e-6)))
    if case["rows"] * case["history"] > 4_000_000:
        return None
    z = st["logits"].double()
    b, v = z.shape
    lens, first = st["lens"].tolist(), st["prompt_lens"].tolist()
    for i in range(b):
        said = st["tokens"][i, : lens[i]].long()
        every = torch.unique(said)
        r = st["repetition"][i].double()
        z[i, every] = torch.minimum(z[i, every] * r, z[i, every] / r)  # r >= 1: the smaller of the two
        words, count = torch.unique(said[first[i]:], return_counts=True)
        z[i, words] -= st["frequency"][i].double() * count + st["presence"][i].double()
        if st["bias"] is not None:
            z[i].index_add_(0, st["bias_ids"][i].long(), st["bias"][i].double())
        if st["mask"] is not None:
            bits = st["mask"][i].long()[torch.arange(v, device="cuda") // 32] >> (torch.arange(v, device="cuda") % 32)
            z[i].masked_fill_(bits % 2 == 0, float("-inf"))
    # the sum is over the values as they are stored; which of two nearly equal values is larger is left to them
    kept = z.to(st["logits"].dtype).double()
    return z, None, torch.logsumexp(kept, 1)
