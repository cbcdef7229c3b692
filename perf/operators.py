"""Measured cases of the training operators beside the optimizer step.

Five operators produce what `muon_adamw_step` consumes, or hold what producing
it needs:

  lookup  rows of an embedding table, scaled
  egrad   the embedding table's gradient from sorted tokens
  pack    an activation held in 8 bits (signed codes, one power of two for
          every 32 features of a token), and read back
  lgrad   a linear layer's weight gradient, dW = dY^T X, from an X held so
  glu     the gated activation h = act(g) u, and its backward pass from g and
          u held so

`run` computes each in plain torch operations, or with `own` through the
package's entry points.  `exact` is the definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

GROUP = 32           # features of a token that share one scale
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one chunk of prompt for the small table of the tiny hybrid model
        {"name": "lookup_tiny", "op": "lookup", "tokens": 37, "vocab": 1000, "hidden": 256,
         "table": "fp32", "out": "fp32"},
        # a training batch through the backbone's token table
        {"name": "lookup_batch", "op": "lookup", "tokens": 65536, "vocab": 151000, "hidden": 2048,
         "table": "bf16", "out": "bf16"},
        # the tiny hybrid model's embedding gradient: latency of a small step
        {"name": "egrad_tiny", "op": "egrad", "tokens": 512, "vocab": 1000, "hidden": 256,
         "dout": "fp32", "grad": "fp32", "pad": False},
        # odd sizes, a padded batch, bf16 activations into fp32 gradients
        {"name": "egrad_ragged", "op": "egrad", "tokens": 50021, "vocab": 32003, "hidden": 1001,
         "dout": "bf16", "grad": "fp32", "pad": True},
        # the backbone's token table when it is trained, stored in bf16
        {"name": "egrad_backbone", "op": "egrad", "tokens": 16384, "vocab": 151000, "hidden": 2048,
         "dout": "bf16", "grad": "bf16", "pad": True},
        # one action chunk of the action expert, kept for its backward pass
        {"name": "pack_chunk", "op": "pack", "rows": 50, "cols": 1024, "dtype": "fp32"},
        # the input of the backbone's down projection over a batch
        {"name": "pack_batch", "op": "pack", "rows": 32768, "cols": 8192, "dtype": "bf16"},
        # tiny hybrid model, fp32 policy, a handful of tokens
        {"name": "lgrad_tiny", "op": "lgrad", "tokens": 77, "n_out": 256, "n_in": 256,
         "dy": "fp32", "grad": "fp32"},
        # k/v projection of the action expert: few outputs, a long token axis
        {"name": "lgrad_kv", "op": "lgrad", "tokens": 16001, "n_out": 256, "n_in": 1024,
         "dy": "bf16", "grad": "fp32"},
        # gate/up projection of the backbone over a batch
        {"name": "lgrad_backbone", "op": "lgrad", "tokens": 32768, "n_out": 8192, "n_in": 2048,
         "dy": "bf16", "grad": "bf16"},
        # one action chunk through the action expert's MLP
        {"name": "glu_chunk", "op": "glu", "rows": 50, "cols": 4096, "act": "gelu_tanh",
         "dtype": "fp32"},
        # the backbone's MLP over a batch
        {"name": "glu_batch", "op": "glu", "rows": 32768, "cols": 8192, "act": "silu",
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, widths, lo, hi):
    """A configured width, or any size of the range."""
    return rng.choice(widths) if rng.random() < 0.5 else _log(rng, lo, hi)


def draw(rng):
    op = rng.choice(["lookup", "egrad", "pack", "lgrad", "glu"])
    kinds = ["bf16", "fp32"]
    if op == "lookup":
        table = rng.choice(kinds)
        return {"op": op, "tokens": _log(rng, 1, 65536), "vocab": _log(rng, 1000, 151000),
                "hidden": _width(rng, [256, 1024, 2048], 33, 2048), "table": table,
                "out": rng.choice(kinds) if table == "fp32" else table}
    if op == "egrad":
        return {"op": op, "tokens": _log(rng, 1, 65536), "vocab": _log(rng, 1000, 151000),
                "hidden": _width(rng, [256, 1024, 2048], 33, 2048), "dout": rng.choice(kinds),
                "grad": rng.choice(kinds), "pad": rng.random() < 0.5}
    if op == "pack":
        kind = rng.choice(kinds)
        return {"op": op, "rows": _log(rng, 1, 32768 if kind == "bf16" else 16384),
                "cols": _width(rng, [256, 1024, 2048, 4096, 8192], 17, 8192), "dtype": kind}
    if op == "lgrad":
        n = _width(rng, [256, 1024, 2048, 4096, 8192], 17, 4096)
        k = _width(rng, [256, 1024, 2048, 4096], 17, 2048)
        dy = rng.choice(["bf16", "bf16", "fp32"])
        most = 32768 * 8192 * 2048 // (8 if dy == "fp32" else 1)
        return {"op": op, "tokens": _log(rng, 1, max(1, min(32768, most // (n * k)))), "n_out": n,
                "n_in": k, "dy": dy, "grad": rng.choice(kinds)}
    kind = rng.choice(kinds)
    return {"op": op, "rows": _log(rng, 1, 32768 if kind == "bf16" else 16384),
            "cols": _width(rng, [256, 1024, 4096, 8192], 17, 8192),
            "act": rng.choice(["silu", "gelu_tanh"]), "dtype": kind}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(DTYPES[dtype])


def _activation(gen, rows, cols, dtype):
    """Activations as layers make them: features of different sizes, a few of
    them far above the others, and token rows that a mask has cleared."""
    size = torch.exp(0.7 * torch.randn(cols, generator=gen, device="cuda"))
    big = torch.rand(cols, generator=gen, device="cuda") < 0.004
    size = torch.where(big, 40.0 * size, size)
    gone = torch.rand(rows, generator=gen, device="cuda") < 0.02
    x = torch.randn((rows, cols), generator=gen, device="cuda") * size
    return x.masked_fill_(gone[:, None], 0.0).to(DTYPES[dtype])


def _token_ids(gen, n, vocab, pad):
    """Tokens of a text: frequencies fall with rank (log-uniform ids), spread
    over the vocabulary; a padded batch ends in its padding token."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab)).to(torch.int64).clamp_(0, vocab - 1)
    ids = (rank * 7919) % vocab
    if pad:
        ids[n - n // 8:] = vocab - 1
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7 + 1)
    s = dict(case)
    op = case["op"]
    if op == "lookup":
        s["w"] = _normal(gen, (case["vocab"], case["hidden"]), 0.02, case["table"])
        s["ids"] = _token_ids(gen, case["tokens"], case["vocab"], False)
        s["scale"] = math.sqrt(case["hidden"])
    elif op == "egrad":
        s["ids"] = _token_ids(gen, case["tokens"], case["vocab"], case["pad"])
        s["d"] = _normal(gen, (case["tokens"], case["hidden"]), 1e-3, case["dout"])
        s["scale"] = math.sqrt(case["hidden"])
        s["skip"] = case["vocab"] - 1 if case["pad"] else -1
    elif op == "pack":
        s["x"] = _activation(gen, case["rows"], case["cols"], case["dtype"])
    elif op == "lgrad":
        x = _activation(gen, case["tokens"], case["n_in"], "bf16")
        s["codes"], s["exps"] = _packed(x)
        s["d"] = _normal(gen, (case["tokens"], case["n_out"]), 1e-3, case["dy"])
    else:
        s["g"] = _activation(gen, case["rows"], case["cols"], case["dtype"]) * 0.5
        s["u"] = _activation(gen, case["rows"], case["cols"], case["dtype"])
        s["d"] = _normal(gen, (case["rows"], case["cols"]), 1e-3, case["dtype"])
    return s


def _packed(x):
    """The stored form of x: codes with rows padded to whole groups, and the
    groups' exponent bytes (2^(e - 127)) with rows padded to whole words."""
    rows, cols = x.shape
    pitch = -(-cols // GROUP) * GROUP
    codes = torch.zeros((rows, pitch), dtype=torch.int8, device=x.device)
    exps = torch.zeros((rows, -(-pitch // GROUP // 4) * 4), dtype=torch.uint8, device=x.device)
    step = max(1, (1 << 26) // pitch)
    for r in range(0, rows, step):
        q, e = _quantise(x[r:r + step].float())
        codes[r:r + step] = q.flatten(1).to(torch.int8)
        exps[r:r + step, :pitch // GROUP] = e.to(torch.uint8)
    return codes, exps


# --------------------------------------------------------------------------
# the operators in plain operations
# --------------------------------------------------------------------------

def _quantise(x):
    """Codes (rows, groups, 32) and exponents (rows, groups) of float32 x: the
    smallest power of two that keeps every rounded quotient within 127."""
    rows, cols = x.shape
    pitch = -(-cols // GROUP) * GROUP
    if pitch != cols:
        x = torch.nn.functional.pad(x, (0, pitch - cols))
    x = x.view(rows, pitch // GROUP, GROUP)
    top = x.abs().amax(2)
    mant, ex = torch.frexp(top)                      # top = mant 2^ex, mant in [1/2, 1)
    e = ex - 7 + (mant * 128.0 >= 127.5).to(ex.dtype)
    e = torch.where(top > 0, e, torch.full_like(e, -126)).clamp_(min=-126)
    return torch.round(torch.ldexp(x, -e[:, :, None])), e + 127


def _held(x):
    """What x is after it was held in 8 bits, in float32."""
    q, e = _quantise(x.float())
    return torch.ldexp(q, e[:, :, None] - 127).flatten(1)[:, :x.shape[1]]


def _from_codes(codes, exps, cols):
    groups = codes.shape[1] // GROUP
    v = codes.view(codes.shape[0], groups, GROUP).float()
    e = exps[:, :groups].to(torch.int32) - 127
    return torch.ldexp(v, e[:, :, None]).flatten(1)[:, :cols]


def _act(kind, g):
    """act(g) and its derivative."""
    if kind == "silu":
        sig = torch.sigmoid(g)
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    c = 2.0 * math.sqrt(2.0 / math.pi)
    sig = torch.sigmoid(c * (g + 0.044715 * g * g * g))
    return g * sig, sig + g * sig * (1.0 - sig) * c * (1.0 + 3 * 0.044715 * g * g)


def run(s):
    op = s["op"]
    if own:
        return _run_own(s)
    if op == "lookup":
        return (s["w"][s["ids"]].float() * s["scale"]).to(DTYPES[s["out"]])
    if op == "egrad":
        src = s["d"].float() * s["scale"]
        src = torch.where((s["ids"] == s["skip"])[:, None], torch.zeros_like(src), src)
        w = torch.zeros((s["vocab"], s["hidden"]), device="cuda")
        return w.index_add_(0, s["ids"], src).to(DTYPES[s["grad"]])
    if op == "pack":
        return _held(s["x"]).to(s["x"].dtype)
    if op == "lgrad":
        x = _from_codes(s["codes"], s["exps"], s["n_in"])
        return torch.matmul(s["d"].float().t(), x).to(DTYPES[s["grad"]])
    g, u, d = s["g"].float(), s["u"].float(), s["d"].float()
    h = _act(s["act"], g)[0] * u
    a, da = _act(s["act"], _held(g))
    to = s["g"].dtype
    return {"h": h.to(to), "dg": (d * _held(u) * da).to(to), "du": (d * a).to(to)}


def _run_own(s):
    import muon_newton_schulz_02_amd as M
    op = s["op"]
    if op == "lookup":
        return M.ma_embedding_lookup(s["w"], s["ids"], scale=s["scale"], out_dtype=DTYPES[s["out"]])
    if op == "egrad":
        return M.ma_embedding_grad(s["d"], s["ids"], s["vocab"], scale=s["scale"],
                                   padding_token=s["skip"], grad_dtype=DTYPES[s["grad"]])
    if op == "pack":
        return M.ma_act_unpack(M.ma_act_pack(s["x"]), s["x"].dtype)
    if op == "lgrad":
        x = M.ActCheckpoint(s["codes"], s["exps"], s["n_in"])
        return M.ma_linear_grad(s["d"], x, grad_dtype=DTYPES[s["grad"]])
    h, g, u = M.ma_glu_forward(s["g"], s["u"], s["act"])
    dg, du = M.ma_glu_backward(s["d"], g, u, s["act"])
    return {"h": h, "dg": dg, "du": du}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def _size(kind):
    return 2 if kind == "bf16" else 4


def _distinct(n, vocab):
    """How many different ids n of _token_ids' are expected to hold."""
    rank = np.arange(1, vocab, dtype=np.float64)
    p = np.log1p(1.0 / rank) / math.log(vocab)
    return int(round(float(-np.expm1(n * np.log1p(-np.minimum(p, 0.999999))).sum())))


def work(case):
    op = case["op"]
    if op == "lookup":
        n = case["tokens"] * case["hidden"]
        rows = max(1, _distinct(case["tokens"], case["vocab"]))       # each read once
        return {"bytes": rows * case["hidden"] * _size(case["table"]) + n * _size(case["out"]) +
                8 * case["tokens"], "flops": n}
    if op == "egrad":
        n = case["tokens"] * case["hidden"]
        kept = n - case["tokens"] // 8 * case["hidden"] if case["pad"] else n
        return {"bytes": kept * _size(case["dout"]) + 8 * case["tokens"] +
                case["vocab"] * case["hidden"] * _size(case["grad"]), "flops": 2 * kept}
    if op == "pack":
        # written in 8 bits and read back: x in, codes out, codes in, values out
        n = case["rows"] * case["cols"]
        held = n + -(-n // GROUP)
        return {"bytes": 2 * n * _size(case["dtype"]) + 2 * held, "flops": 4 * n}
    if op == "lgrad":
        m, n, k = case["tokens"], case["n_out"], case["n_in"]
        return {"bytes": m * n * _size(case["dy"]) + m * k + -(-m * k // GROUP) +
                n * k * _size(case["grad"]), "flops": 2 * m * n * k}
    # g, u in, h and both held forms out; d and both held forms in, dg, du out
    n = case["rows"] * case["cols"]
    held = n + -(-n // GROUP)
    return {"bytes": 6 * n * _size(case["dtype"]) + 4 * held, "flops": 30 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _held64(x):
    """x after 8 bits, from the definition: the scale is the smallest 2^k, k
    from -126, for which no |x| / 2^k of the group rounds above 127."""
    rows, cols = x.shape
    out = torch.empty((rows, cols), dtype=torch.float64, device=x.device)
    step = max(1, (1 << 25) // cols)
    for r in range(0, rows, step):
        v = x[r:r + step].double()
        whole = cols // GROUP * GROUP
        parts = [v[:, :whole].reshape(-1, GROUP)] if whole else []
        if whole < cols:
            parts.append(v[:, whole:])
        got = []
        for p in parts:
            top = p.abs().amax(1, keepdim=True)
            k = torch.floor(torch.log2(top / 127.0)).clamp(min=-126.0) - 1.0
            for _ in range(3):      # up to the first scale that holds the group
                k = torch.where(torch.round(top * torch.exp2(-k)) > 127.0, k + 1.0, k)
            k = k.clamp(min=-126.0)
            got.append(torch.round(p * torch.exp2(-k)) * torch.exp2(k))
        if whole:
            out[r:r + step, :whole] = got[0].reshape(v.shape[0], whole)
        if whole < cols:
            out[r:r + step, whole:] = got[-1]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        return torch.index_select(s["w"], 0, s["ids"]).double().mul_(s["scale"])
    if op == "egrad":
        keep = s["ids"] != s["skip"]
        ids, order = torch.sort(s["ids"][keep], stable=True)
        w = torch.zeros((case["vocab"], case["hidden"]), dtype=torch.float64, device="cuda")
        if ids.numel():
            total = torch.cumsum(s["d"][keep][order].double(), 0)
            last = torch.cat([ids[1:] != ids[:-1], torch.ones(1, dtype=torch.bool, device="cuda")])
            ends = total[last]
            w[ids[last]] = torch.diff(ends, dim=0, prepend=torch.zeros_like(ends[:1])) * s["scale"]
        return w
    if op == "pack":
        return _held64(s["x"])
    if op == "lgrad":
        two = torch.exp2(s["exps"].double() - 127.0)[:, :s["codes"].shape[1] // GROUP]
        x = (s["codes"].double() * two.repeat_interleave(GROUP, 1))[:, :case["n_in"]]
        w = torch.zeros((case["n_out"], case["n_in"]), dtype=torch.float64, device="cuda")
        step = 4096
        for t in range(0, case["tokens"], step):
            w += s["d"][t:t + step].double().t().contiguous() @ x[t:t + step]
        return w
    g, u, d = s["g"].double(), s["u"].double(), s["d"].double()

    def act(v):
        if case["act"] == "silu":
            return v / (1.0 + torch.exp(-v))
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))

    def slope(v):
        if case["act"] == "silu":
            e = torch.exp(-v.abs())
            p = torch.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
            return p + v * e / (1.0 + e) ** 2
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * v * v)

    gh, uh = _held64(s["g"]), _held64(s["u"])
    return {"h": act(g) * u, "dg": d * uh * slope(gh), "du": d * act(gh)}
