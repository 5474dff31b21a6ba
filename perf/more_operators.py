"""What is measured of the operators that close the loop from a token to the next one: the embedding of the
ids with its gradient, the head's product on 4-bit weights, and the choice of a token from its logits.

``run`` computes each in elementary torch operations, or, where ``own`` is true, by the calls that a
user of the package makes.  ``exact`` is each operator's definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32  # columns that share a scale in the 4-bit format


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------
def listed():
    return [
        # the last tokens of eight requests enter the model: latency
        {"name": "embed-decode-8", "op": "embed", "tokens": 8, "vocab": 151936, "cols": 4096, "dtype": "bf16",
         "out": "bf16", "scale": 1.0, "ids32": False},
        # a training step's 16384 tokens, scaled by the root of the width, into an fp32 residual stream
        {"name": "embed-train", "op": "embed", "tokens": 16384, "vocab": 151936, "cols": 4096, "dtype": "bf16",
         "out": "f32", "scale": 64.0, "ids32": False},
        # the table's gradient of that step: all 151936 rows are written
        {"name": "embed-bwd-train", "op": "embed-bwd", "tokens": 16384, "vocab": 151936, "cols": 4096,
         "dtype": "bf16", "out": "bf16", "scale": 64.0, "ids32": False},
        # a ragged batch over a small fp32 table of odd width: long runs of the same few words
        {"name": "embed-bwd-ragged", "op": "embed-bwd", "tokens": 20011, "vocab": 4099, "cols": 1283, "dtype": "f32",
         "out": "f32", "scale": 1.0, "ids32": True},
        # a head's weight taken to 4 bits once, and looked at again in 16 bits
        {"name": "mx4-weight", "op": "mx4", "rows": 128256, "cols": 2048, "dtype": "bf16"},
        # fp32 activations of an odd width to 4 bits and back
        {"name": "mx4-rows-odd", "op": "mx4", "rows": 301, "cols": 1283, "dtype": "f32"},
        # one request's logits from a 4-bit head: the weight's bytes count
        {"name": "mx4-logits-1", "op": "mx4-logits", "tokens": 1, "vocab": 151936, "cols": 4096, "dtype": "bf16",
         "out": "bf16", "bias": False, "scale": 1.0, "cap": 0.0},
        # a serving batch, with bias, scale and soft cap, logits in fp32
        {"name": "mx4-logits-64", "op": "mx4-logits", "tokens": 64, "vocab": 128256, "cols": 2048, "dtype": "bf16",
         "out": "f32", "bias": True, "scale": 0.25, "cap": 30.0},
        # scoring a text: the logits of 2047 positions
        {"name": "mx4-logits-2047", "op": "mx4-logits", "tokens": 2047, "vocab": 151936, "cols": 4096,
         "dtype": "bf16", "out": "bf16", "bias": False, "scale": 1.0, "cap": 0.0},
        # one request's next token with the filters that a chat uses
        {"name": "sample-1", "op": "sample", "rows": 1, "vocab": 151936, "dtype": "f32", "filters": "chat"},
        # a serving batch of requests with settings of their own, greedy ones among them
        {"name": "sample-mixed-61", "op": "sample", "rows": 61, "vocab": 100003, "dtype": "f16", "filters": "mixed"},
        # the largest batch: a nucleus of a 262144-word vocabulary
        {"name": "sample-nucleus-256", "op": "sample", "rows": 256, "vocab": 262144, "dtype": "f32",
         "filters": "nucleus"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A size between lo and hi: a multiple of 128, of 8, or any."""
    step = rng.choice([128, 8, 8, 1])
    return max(lo, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["embed", "embed-bwd", "embed-bwd", "mx4", "mx4-logits", "mx4-logits", "sample", "sample"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("embed", "embed-bwd"):
        cols = _width(rng, 64, 8192)
        vocab = _width(rng, 1000, min(262144, 151936 * 4096 // cols))
        tokens = _log_int(rng, 1, min(32768, 16384 * 4096 // cols))
        return {"op": op, "tokens": tokens, "vocab": vocab, "cols": cols, "dtype": dtype,
                "out": rng.choice([dtype, dtype, "f32"]), "scale": rng.choice([1.0, 1.0, math.sqrt(cols)]),
                "ids32": rng.random() < 0.5}
    if op == "mx4":
        cols = _width(rng, 33, 16384)
        return {"op": op, "rows": _log_int(rng, 1, min(262144, 128256 * 2048 // cols)), "cols": cols, "dtype": dtype}
    if op == "mx4-logits":
        cols = _width(rng, 64, 8192)
        vocab = _width(rng, 1000, min(262144, 151936 * 4096 // cols))
        return {"op": op, "tokens": _log_int(rng, 1, 2047), "vocab": vocab, "cols": cols, "dtype": dtype,
                "out": rng.choice(["bf16", "f16", "f32"]), "bias": rng.random() < 0.5,
                "scale": rng.choice([1.0, 0.25]), "cap": rng.choice([0.0, 0.0, 30.0])}
    return {"op": op, "rows": _log_int(rng, 1, 256), "vocab": _width(rng, 1000, 262144), "dtype": dtype,
            "filters": rng.choice(["none", "chat", "mixed", "mixed", "nucleus"])}


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kw = dict(generator=g, device="cuda", dtype=torch.float32)
    st = {"case": case}
    op = case["op"]
    if op in ("embed", "embed-bwd"):
        n, v, d = case["tokens"], case["vocab"], case["cols"]
        # texts repeat a few words often; the end of a padded batch has no word
        ids = (v * torch.rand(n, generator=g, device="cuda", dtype=torch.float64).pow(3)).long().clamp_(max=v - 1)
        ids[n - n // 16:] = -1
        st["ids"] = ids.to(torch.int32 if case["ids32"] else torch.int64)
        if op == "embed":
            st["weight"] = (torch.randn(v, d, **kw) * 0.02).to(DTYPES[case["dtype"]])
        else:
            st["dout"] = (torch.randn(n, d, **kw) * 1e-3).to(DTYPES[case["out"]])
        return st
    if op == "mx4":
        # columns differ in size, and a few values by far
        x = torch.randn(case["rows"], case["cols"], **kw)
        x *= torch.exp(torch.randn(case["cols"], **kw))
        st["x"] = x.to(DTYPES[case["dtype"]])
        return st
    if op == "mx4-logits":
        n, v, d = case["tokens"], case["vocab"], case["cols"]
        st["hidden"] = (torch.randn(n, d, **kw) * torch.exp(0.5 * torch.randn(d, **kw))).to(DTYPES[case["dtype"]])
        grid, power = _mx4(torch.randn(v, d, **kw) * (2.0 / math.sqrt(d)))
        # what a program keeps of its weight: the packed codes and scales, and for the plain form its values
        st["codes"], st["scales"] = _packed(grid, power)
        st["weight"] = (grid * _pow2(power)[..., None]).view(v, -1)[:, :d].contiguous()
        st["bias"] = torch.randn(v, **kw).to(DTYPES[case["dtype"]]) if case["bias"] else None
        return st
    b, v = case["rows"], case["vocab"]
    z = torch.randn(b, v, **kw) * 3.0
    z[:, v - 1 - v // 50:] = float("-inf")  # the padding of the vocabulary
    row = torch.arange(b, device="cuda")
    z[row % 32 == 31] = float("-inf")       # a grammar at its end: nothing is allowed
    st["logits"] = z.to(DTYPES[case["dtype"]])
    st["uniform"] = torch.rand(b, **kw)
    st["temperature"] = st["top_k"] = st["top_p"] = st["min_p"] = None
    pick = lambda *x: torch.tensor(x, device="cuda")[torch.randint(0, len(x), (b,), generator=g, device="cuda")]  # noqa: E731
    if case["filters"] == "chat":
        st["temperature"], st["top_k"] = torch.full((b,), 0.8, device="cuda"), torch.full((b,), 50, device="cuda")
        st["top_p"] = torch.full((b,), 0.95, device="cuda")
    elif case["filters"] == "nucleus":
        st["temperature"], st["top_p"] = pick(0.7, 0.9, 1.0), pick(0.8, 0.9, 0.95)
    elif case["filters"] == "mixed":
        st["temperature"], st["top_k"] = pick(0.0, 0.6, 0.8, 1.0, 1.3), pick(0, 0, 1, 40, 1000, 20000)
        st["top_p"], st["min_p"] = pick(1.0, 0.5, 0.9, 0.99), pick(0.0, 0.0, 0.02, 0.1)
    return st


def _mx4(x):
    """fp32 rows as [rows, blocks, 32] values of the 4-bit grid and [rows, blocks] powers of two."""
    n, d = x.shape
    blocks = -(-d // BLOCK)
    x = torch.nn.functional.pad(x, (0, blocks * BLOCK - d)).view(n, blocks, BLOCK)
    top = x.abs().amax(2)
    power = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 125)
    y = x * _pow2(-power)[..., None]
    a = y.abs()
    # steps of 1/2 to 2, of 1 to 4, of 2 above; halves go to the even code
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.copysign(a, y), power


def _pow2(k):
    """2^k for -127 <= k <= 127, from its bits."""
    return torch.where(k > -127, (k + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _packed(grid, power):
    """The codes, two to a byte (the even column in the low half), and the scales' exponents + 127 in tiles of
    128 rows x 4 blocks, in which row r is entry (r % 32, r // 32)."""
    n, blocks, _ = grid.shape
    a = grid.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code += torch.signbit(grid).to(torch.uint8) * 8
    codes = (code[..., 0::2] + code[..., 1::2] * 16).view(n, blocks * (BLOCK // 2))
    nt, kt = -(-n // 128), -(-blocks // 4)
    s = torch.nn.functional.pad((power + 127).to(torch.uint8), (0, kt * 4 - blocks, 0, nt * 128 - n))
    return codes, s.view(nt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous()


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------
def run(st):
    case = st["case"]
    if own:
        return _run_own(case, st)
    if case["op"] == "embed":
        return _plain_embed(case, st)
    if case["op"] == "embed-bwd":
        return _plain_embed_bwd(case, st)
    if case["op"] == "mx4":
        grid, power = _mx4(st["x"].float())
        return (grid * _pow2(power)[..., None]).view(case["rows"], -1)[:, :case["cols"]].to(st["x"].dtype)
    if case["op"] == "mx4-logits":
        return _plain_logits(case, st)
    return _plain_sample(st)


def _run_own(case, st):
    import linear_cross_entropy_tmem_gb300 as flce
    if case["op"] == "embed":
        return flce.flce_embedding(st["weight"], st["ids"], scale=case["scale"], out_dtype=DTYPES[case["out"]])
    if case["op"] == "embed-bwd":
        return flce.flce_embedding_backward(st["dout"], st["ids"], case["vocab"], scale=case["scale"],
                                            dtype=DTYPES[case["dtype"]])
    if case["op"] == "mx4":
        return flce.mxfp4_dequantize(flce.mxfp4_quantize(st["x"]), st["x"].dtype)
    if case["op"] == "mx4-logits":
        return flce.mxfp4_logits(st["hidden"], flce.MxFp4(st["codes"], st["scales"], case["cols"]), st["bias"],
                                 logit_scale=case["scale"], softcap=case["cap"], out_dtype=DTYPES[case["out"]])
    r = flce.sample_tokens(st["logits"], st["uniform"], temperature=st["temperature"], top_k=st["top_k"],
                           top_p=st["top_p"], min_p=st["min_p"])
    return r.token, r.logprob, r.kept


def _plain_embed(case, st):
    ids = st["ids"].long()
    there = (ids >= 0) & (ids < case["vocab"])
    rows = st["weight"][ids.clamp(0, case["vocab"] - 1)].float() * case["scale"]
    return torch.where(there[:, None], rows, torch.zeros_like(rows)).to(DTYPES[case["out"]])


def _plain_embed_bwd(case, st):
    ids = st["ids"].long()
    there = (ids >= 0) & (ids < case["vocab"])
    rows = torch.where(there[:, None], st["dout"].float(), 0.0)
    dw = torch.zeros(case["vocab"], case["cols"], dtype=torch.float32, device=rows.device)
    dw.index_add_(0, ids.clamp(0, case["vocab"] - 1), rows)
    return dw.mul_(case["scale"]).to(DTYPES[case["dtype"]])


def _plain_logits(case, st):
    grid, power = _mx4(st["hidden"].float())
    h = (grid * _pow2(power)[..., None]).view(case["tokens"], -1)[:, :case["cols"]]
    z = h @ st["weight"].t()
    if st["bias"] is not None:
        z += st["bias"].float()
    z *= case["scale"]
    if case["cap"]:
        z = torch.tanh(z / case["cap"]) * case["cap"]
    return z.to(DTYPES[case["out"]])


def _plain_sample(st):
    z = st["logits"].double()
    b, v = z.shape
    full = lambda x, default: torch.full((b, 1), default, dtype=torch.float64, device=z.device) if x is None \
        else x[:, None].double()  # noqa: E731
    t, k = full(st["temperature"], 1.0), full(st["top_k"], 0.0)
    p, least = full(st["top_p"], 1.0), full(st["min_p"], 0.0)
    k = torch.where(k > 0, k, float(v))
    k, t = torch.where(t > 0, k, 1.0), torch.where(t > 0, t, 1.0)  # greedy: the first of the largest
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    top = zs[:, :1]
    some = top > float("-inf")
    ws = torch.where(some, torch.exp((zs - top) / t), torch.zeros_like(zs))
    ws = torch.where(torch.arange(v, device=z.device)[None] < k, ws, torch.zeros_like(ws))
    upto = ws.cumsum(1)
    # the nucleus: entries before which less than p of the mass lies, the first one always
    keep = (ws > 0) & (ws >= least) & ((p >= 1) | (upto - ws < p * upto[:, -1:]))
    keep[:, :1] |= some
    w = torch.zeros_like(ws).scatter_(1, order, torch.where(keep, ws, torch.zeros_like(ws)))
    upto = w.cumsum(1)
    mass = upto[:, -1:]
    last = torch.where(w > 0, torch.arange(v, device=z.device)[None], -1).amax(1)
    token = torch.minimum((upto <= st["uniform"][:, None].double() * mass).sum(1), last)
    mine = w.gather(1, token.clamp(min=0)[:, None])
    logprob = torch.where(some, torch.log(mine / mass), float("-inf"))[:, 0]
    return token, logprob.float(), (w > 0).sum(1)


# ---------------------------------------------------------------------------------------------------
# Work, and the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("embed", "embed-bwd"):
        n, v, d = case["tokens"], case["vocab"], case["cols"]
        ids = n * (4 if case["ids32"] else 8)
        if op == "embed":
            return {"bytes": ids + n * d * (BYTES[case["dtype"]] + BYTES[case["out"]]), "flops": 1.0 * n * d}
        return {"bytes": ids + n * d * BYTES[case["out"]] + v * d * BYTES[case["dtype"]], "flops": 1.0 * n * d}
    if op == "mx4":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * BYTES[case["dtype"]] + 2 * n * 17 / 32, "flops": 4.0 * n}
    if op == "mx4-logits":
        n, v, d = case["tokens"], case["vocab"], case["cols"]
        return {"bytes": v * d * 17 / 32 + n * d * BYTES[case["dtype"]] + n * v * BYTES[case["out"]]
                + (v * BYTES[case["dtype"]] if case["bias"] else 0), "flops": 2.0 * n * v * d}
    return {"bytes": case["rows"] * (case["vocab"] * BYTES[case["dtype"]] + 44),
            "flops": 8.0 * case["rows"] * case["vocab"]}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        ids = st["ids"].long()
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(ids >= 0).squeeze(1)
        out[at] = torch.index_select(st["weight"], 0, ids[at]).double().mul(case["scale"])
        return out
    if op == "embed-bwd":
        ids = st["ids"].long()
        at = torch.nonzero(ids >= 0).squeeze(1)
        dw = torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device="cuda")
        return dw.index_put_((ids[at],), st["dout"][at].double() * case["scale"], accumulate=True)
    if op == "mx4":
        return _nearest(st["x"].double())
    if op == "mx4-logits":
        v, d = case["vocab"], case["cols"]
        value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                             device="cuda")
        c = st["codes"].int()
        w = torch.stack([value[c & 15], value[c >> 4]], 2).view(v, -1, BLOCK)
        r, k = torch.arange(v, device="cuda")[:, None], torch.arange(w.shape[1], device="cuda")[None]
        w *= torch.exp2(st["scales"][r // 128, k // 4, r % 32, r % 128 // 32, k % 4].double() - 127).unsqueeze(2)
        z = torch.einsum("nd,vd->nv", _nearest(st["hidden"].double()), w.view(v, -1)[:, :d])
        if st["bias"] is not None:
            z = z + st["bias"].double()
        z = z * case["scale"]
        return case["cap"] * torch.tanh(z / case["cap"]) if case["cap"] else z
    if case["rows"] * case["vocab"] > 80_000_000:
        return None
    return None, _logprobs(st), None


def _nearest(x):
    """Each value's nearest of the 4-bit grid at its block's scale, by the borders between the grid's values."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    low = torch.tensor([.25, 1.25, 2.5, 5], dtype=torch.float64, device=x.device)   # a border itself goes down
    high = torch.tensor([.75, 1.75, 3.5], dtype=torch.float64, device=x.device)     # a border itself goes up
    out = []
    for part in x.split(BLOCK, dim=1):
        top = part.abs().amax(1, keepdim=True)
        # (the addend is far below the distance of an fp32 value from a power of two)
        scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300)) + 1e-9).sub(2).clamp(-127, 125))
        a = part.abs() / scale
        i = torch.bucketize(a, low) + torch.bucketize(a, high, right=True)
        out.append(torch.sign(part) * grid[i] * scale)
    return torch.cat(out, 1)


def _logprobs(st):
    """The chosen token's log-probability among the kept ones, row by row."""
    got = []
    for i in range(st["logits"].shape[0]):
        z = st["logits"][i].double()
        n = int((z > float("-inf")).sum())
        t = 1.0 if st["temperature"] is None else float(st["temperature"][i])
        if n == 0 or t <= 0:
            got.append(float("-inf") if n == 0 else 0.0)
            continue
        by = torch.argsort(z, descending=True, stable=True)[:n]
        if st["top_k"] is not None and int(st["top_k"][i]) > 0:
            by = by[:int(st["top_k"][i])]
        q = torch.softmax(z[by] / t, 0)
        keep = torch.ones_like(q, dtype=torch.bool)
        if st["top_p"] is not None and float(st["top_p"][i]) < 1:
            keep[1:] &= q.cumsum(0)[:-1] < float(st["top_p"][i])
        if st["min_p"] is not None:
            keep[1:] &= (q[1:] / q[0]) >= float(st["min_p"][i])
        by = by[keep].sort().values
        q = torch.softmax(z[by] / t, 0)
        at = int((q.cumsum(0) <= float(st["uniform"][i])).sum().clamp(max=len(by) - 1))
        got.append(float(torch.log(q[at])))
    return torch.tensor(got, dtype=torch.float64)
