"""The operators around the binarized linears of a training step, as measured work.

Embeddings and layer norms of a binarized model stay in full precision; training one needs
their gradients next to the straight-through gradients of the linears, and a global gradient
norm over all of them:

* ``ln``        layer norm forward: y, and the row means and reciprocal deviations for training
* ``ln_bwd``    its gradient: dx, and dweight and dbias reduced over the tokens
* ``embed``     embedding rows of the tokens, times a scale
* ``embed_bwd`` the gradient of the whole table: the rows of dy added up by token, zeros elsewhere
* ``clip``      the 2-norm over many gradient tensors and the gradients scaled down to a largest norm

A case is a dict of plain values, ``prepare`` makes its inputs from a seed, ``run`` makes one pass:
in elementary torch operations, or with ``own`` through the library. ``exact`` states the same
results in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-5

# one 7B-shaped decoder layer: q, k, v, o, gate, up, down as (outputs, inputs)
LAYER_7B = [(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]


def listed():
    return [
        # one token of a 7B-shaped model being decoded: the norm ahead of its projections
        {"name": "ln_1x4096", "op": "ln", "M": 1, "K": 4096, "x": "bf16", "y": "bf16", "affine": True, "stats": False},
        # a training batch at that width, statistics kept for the gradient
        {"name": "ln_4096x4096", "op": "ln", "M": 4096, "K": 4096, "x": "bf16", "y": "bf16", "affine": True,
         "stats": True},
        # a residual stream held in fp32, of an odd width, normed into the linears' bf16
        {"name": "ln_1537x5001_f32", "op": "ln", "M": 1537, "K": 5001, "x": "f32", "y": "bf16", "affine": True,
         "stats": True},
        # the gradient at one sequence of the 7B shape
        {"name": "ln_bwd_2048x4096", "op": "ln_bwd", "M": 2048, "K": 4096, "x": "bf16", "y": "bf16", "affine": True},
        # the gradient over a large batch at the 1.3B width, residual stream in fp32
        {"name": "ln_bwd_16384x2048_f32", "op": "ln_bwd", "M": 16384, "K": 2048, "x": "f32", "y": "bf16",
         "affine": True},
        # a short ragged batch of an odd width
        {"name": "ln_bwd_777x1001", "op": "ln_bwd", "M": 777, "K": 1001, "x": "bf16", "y": "bf16", "affine": True},
        # a decode batch of 16 requests: the rows of their last tokens
        {"name": "embed_16x4096", "op": "embed", "T": 16, "V": 32000, "D": 4096, "table": "bf16", "y": "bf16",
         "ids": "i64", "pad": 0.0},
        # a training batch read out of the fp32 master table, scaled by sqrt(D)
        {"name": "embed_16384x2048", "op": "embed", "T": 16384, "V": 32000, "D": 2048, "table": "f32", "y": "bf16",
         "ids": "i64", "pad": 0.1},
        # the table's gradient for one sequence: most rows are zeros
        {"name": "embed_bwd_2048x2048", "op": "embed_bwd", "T": 2048, "V": 32000, "D": 2048, "table": "f32",
         "y": "bf16", "ids": "i64", "pad": 0.0},
        # ... and for a large padded batch of the 7B width: frequent tokens come up thousands of times
        {"name": "embed_bwd_32768x4096", "op": "embed_bwd", "T": 32768, "V": 32000, "D": 4096, "table": "f32",
         "y": "bf16", "ids": "i32", "pad": 0.15},
        # the gradients of a small model: many tensors of uneven sizes in one flat buffer
        {"name": "clip_small_180", "op": "clip", "kind": "ragged", "count": 180, "total": 6000000, "g": "f32",
         "layout": 3, "max_norm": 1.0},
        # the fp32 gradients of one 7B-shaped layer: seven weights, their scales, two norms
        {"name": "clip_layer_7b", "op": "clip", "kind": "layer_7b", "count": 18, "total": 202434048, "g": "f32",
         "layout": 0, "max_norm": 1.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: as often a multiple of 128 as any number, odd ones among them."""
    k = _log_int(rng, lo, hi)
    return max(128, k // 128 * 128) if rng.random() < 0.5 else k


def draw(rng):
    op = rng.choice(["ln", "ln_bwd", "embed", "embed_bwd", "clip"])
    x, y = rng.choice(["bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"])
    if op in ("ln", "ln_bwd"):
        K = _width(rng, 64, 16384)
        M = _log_int(rng, 1, max(1, min(65536, (1 << 26) // K)))
        c = {"op": op, "M": M, "K": K, "x": x, "y": y, "affine": rng.random() < 0.8}
        return dict(c, stats=rng.random() < 0.6) if op == "ln" else c
    if op in ("embed", "embed_bwd"):
        D = _width(rng, 64, 8192)
        V = _log_int(rng, 256, max(256, min(131072, (1 << 27) // D)))
        T = _log_int(rng, 1, max(1, min(65536, (1 << 27) // D)))
        return {"op": op, "T": T, "V": V, "D": D, "table": x, "y": y, "ids": rng.choice(["i32", "i64"]),
                "pad": rng.choice([0.0, 0.0, 0.2, 0.6])}
    count = _log_int(rng, 1, 400)
    return {"op": "clip", "kind": "ragged", "count": count, "total": _log_int(rng, max(1000, count), 100000000), "g": x,
            "layout": rng.randrange(1 << 20), "max_norm": rng.choice([1.0, 0.25, 1e6])}


def _sizes(case):
    """Numbers of elements of a clip case's tensors."""
    if case["kind"] == "layer_7b":
        return [n * k for n, k in LAYER_7B] + [n for n, _ in LAYER_7B] + [4096] * 4
    rng = random.Random(case["layout"])
    share = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(case["count"])]
    unit = case["total"] / sum(share)
    return [max(1, int(s * unit)) for s in share]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ids(case, g):
    """Tokens by Zipf's law over a shuffled vocabulary; the last rows of the batch are padding (id 0)."""
    T, V = case["T"], case["V"]
    p = 1.0 / (torch.arange(V, device="cuda", dtype=torch.float64) + 2.7)
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * p.sum()
    rank = torch.searchsorted(p.cumsum(0), u).clamp_(max=V - 1)
    ids = torch.randperm(V, generator=g, device="cuda")[rank]
    ids[T - int(case["pad"] * T):] = 0
    return ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"op": op}
    if op in ("ln", "ln_bwd"):
        M, K = case["M"], case["K"]
        # activations with an offset and a spread for each channel, a few channels far out
        x = randn(M, K) * (1.0 + 0.5 * randn(K).abs()) + 0.3 * randn(K)
        x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 10.0
        s["x"] = x.to(TYPES[case["x"]])
        del x
        s["weight"] = 1.0 + 0.1 * randn(K) if case["affine"] else None
        s["bias"] = 0.1 * randn(K) if case["affine"] else None
        s["y_type"] = TYPES[case["y"]]
        if op == "ln":
            s["stats"] = case["stats"]
        else:
            # what the forward pass kept
            m = s["x"].mean(1, dtype=torch.float64)
            v = s["x"].double().sub_(m[:, None]).square_().mean(1)
            s["mean"], s["rstd"] = m.float(), (v + EPS).rsqrt().float()
            s["dy"] = (0.01 * randn(M, K)).to(TYPES[case["y"]])
    elif op in ("embed", "embed_bwd"):
        s["ids"] = _ids(case, g)
        s["V"], s["scale"] = case["V"], math.sqrt(case["D"])
        if op == "embed":
            s["table"] = (0.02 * randn(case["V"], case["D"])).to(TYPES[case["table"]])
            s["y_type"] = TYPES[case["y"]]
        else:
            s["dy"] = (0.01 * randn(case["T"], case["D"])).to(TYPES[case["y"]])
            s["table_type"] = TYPES[case["table"]]
            s["padding_id"] = 0 if case["pad"] else None
    else:
        sizes = _sizes(case)
        n = sum(sizes)
        flat = randn(n)
        at = 0
        for i, k in enumerate(sizes):  # tensors differ in scale by a few powers of ten
            flat[at:at + k] *= 10.0 ** (-2 - i % 3)
            at += k
        s["flat"] = flat.to(TYPES[case["g"]])
        s["out"] = torch.empty_like(s["flat"])
        s["grads"], s["outs"] = list(s["flat"].split(sizes)), list(s["out"].split(sizes))
        s["max_norm"] = case["max_norm"]
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_plain(s):
    op = s["op"]
    if op == "ln":
        x = s["x"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).mean(1) + EPS)
        y = d * rstd[:, None]
        if s["weight"] is not None:
            y = y * s["weight"] + s["bias"]
        y = y.to(s["y_type"])
        return {"y": y, "mean": mean, "rstd": rstd} if s["stats"] else {"y": y}
    if op == "ln_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy if s["weight"] is None else dy * s["weight"]
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        out = {"dx": dx.to(s["x"].dtype)}
        if s["weight"] is not None:
            out["dweight"], out["dbias"] = (dy * xhat).sum(0), dy.sum(0)
        return out
    if op == "embed":
        return {"y": (s["table"][s["ids"].long()].float() * s["scale"]).to(s["y_type"])}
    if op == "embed_bwd":
        ids, dy = s["ids"].long(), s["dy"].float() * s["scale"]
        if s["padding_id"] is not None:
            dy = dy * (ids != s["padding_id"])[:, None]
        d = torch.zeros(s["V"], dy.shape[1], device=dy.device).index_add_(0, ids, dy)
        return {"dtable": d.to(s["table_type"])}
    # the flat buffer holds every tensor: one sum and one product serve them all
    norm = s["flat"].double().square().sum().sqrt()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm.float(), "coef": coef.float(), "grads": (s["flat"].float() * coef.float()).to(s["flat"].dtype)}


def _run_own(s):
    import bit_linear_layers_b200 as bl
    op = s["op"]
    if op == "ln":
        got = bl.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, out_dtype=s["y_type"], stats=s["stats"])
        return {"y": got[0], "mean": got[1], "rstd": got[2]} if s["stats"] else {"y": got}
    if op == "ln_bwd":
        dx, dw, db = bl.layer_norm_backward(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"],
                                            want_dw=s["weight"] is not None)
        return {"dx": dx} if s["weight"] is None else {"dx": dx, "dweight": dw, "dbias": db}
    if op == "embed":
        return {"y": bl.embedding(s["ids"], s["table"], scale=s["scale"], out_dtype=s["y_type"])}
    if op == "embed_bwd":
        return {"dtable": bl.embedding_backward(s["ids"], s["dy"], s["V"], scale=s["scale"],
                                                padding_id=s["padding_id"], out_dtype=s["table_type"])}
    norm, coef = bl.grad_clip(s["grads"], s["max_norm"], out=s["outs"])
    return {"norm": norm, "coef": coef, "grads": s["out"]}


def work(case):
    op = case["op"]
    if op in ("ln", "ln_bwd"):
        M, K, bx, by = case["M"], case["K"], BYTES[case["x"]], BYTES[case["y"]]
        affine = 8 * K if case["affine"] else 0
        if op == "ln":
            return {"bytes": M * K * (bx + by) + affine + (8 * M if case["stats"] else 0), "flops": 8 * M * K}
        # x, dy and dx; the weight and the statistics; dweight and dbias
        return {"bytes": M * K * (2 * bx + by) + 8 * M + 1.5 * affine, "flops": 14 * M * K}
    if op in ("embed", "embed_bwd"):
        T, V, D, bi = case["T"], case["V"], case["D"], 4 if case["ids"] == "i32" else 8
        bt, by = BYTES[case["table"]], BYTES[case["y"]]
        if op == "embed":
            # a row that several tokens share is read once: the expected number of distinct tokens by Zipf's law
            return {"bytes": T * bi + _distinct(case) * D * bt + T * D * by, "flops": T * D}
        live = T - (int(case["pad"] * T) if case["pad"] else 0)
        return {"bytes": T * bi + live * D * by + V * D * bt, "flops": 2 * live * D}
    n = sum(_sizes(case))
    return {"bytes": 2 * n * BYTES[case["g"]] + 8, "flops": 3 * n}


def _distinct(case):
    T, V = case["T"] - int(case["pad"] * case["T"]), case["V"]
    z = sum(1.0 / (v + 2.7) for v in range(V))
    return sum(-math.expm1(T * math.log1p(-1.0 / ((v + 2.7) * z))) for v in range(V)) + (1 if case["pad"] else 0)


def exact(case, seed):
    """The definitions in fp64."""
    s, op = prepare(case, seed), case["op"]
    if op == "ln":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        y = x.sub_(mean[:, None]).div_((var + EPS).sqrt()[:, None])
        if s["weight"] is not None:
            y = torch.addcmul(s["bias"].double(), y, s["weight"].double())
        return {"y": y, "mean": mean, "rstd": (var + EPS) ** -0.5} if s["stats"] else {"y": y}
    if op == "ln_bwd":
        # the statistics are the rows' own, not the kept roundings of them
        x, dy = s["x"].double(), s["dy"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        root = (var + EPS).sqrt()[:, None]
        z = x.sub_(mean[:, None]).div_(root)
        out = {"dx": None}
        if s["weight"] is not None:
            out["dweight"], out["dbias"] = torch.einsum("mk,mk->k", dy, z), torch.einsum("mk->k", dy)
            dy = dy * s["weight"].double()
        K = dy.shape[1]
        along = torch.einsum("mk,mk->m", dy, z)[:, None] / K
        out["dx"] = (dy - dy.sum(1, keepdim=True) / K - along * z) / root
        return out
    if op == "embed":
        return {"y": torch.index_select(s["table"].double(), 0, s["ids"].long()) * s["scale"]}
    if op == "embed_bwd":
        # tokens in order of their ids; a row's sum is a difference of running sums
        ids = s["ids"].long()
        order = torch.argsort(ids, stable=True)
        if s["padding_id"] is not None:
            order = order[ids[order] != s["padding_id"]]
        d = torch.zeros(s["V"], case["D"], dtype=torch.float64, device="cuda")
        if order.numel():
            rows, n = torch.unique_consecutive(ids[order], return_counts=True)
            run_sum = torch.cat([torch.zeros(1, case["D"], dtype=torch.float64, device="cuda"),
                                 s["dy"][order].double().cumsum(0)])
            end = n.cumsum(0)
            d[rows] = (run_sum[end] - run_sum[end - n]) * s["scale"]
        return {"dtable": d}
    flat = s["flat"].double()
    norm = torch.linalg.vector_norm(flat)
    coef = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
    return {"norm": norm, "coef": torch.tensor(coef, dtype=torch.float64), "grads": flat * coef}
