"""What stands between the products of a ternary decoder layer, and a layer of experts: cases, inputs and plain forms.

Four operators:

* ``norm``: the residual stream's addition (or the gated sum of what a token's experts gave), the root-mean-square norm
  and the per-token int8 quantisation, as the next product takes them;
* ``linear``: the W2A8 product with bias, activation (gated or not) and residual in its epilogue;
* ``grouped``: that product by expert, rows gathered from the tokens, ragged numbers of rows;
* ``route``: the experts of each token from the router's logits, their gates, and the sorted plan that ``grouped`` and
  ``norm`` read.

``run`` computes each of them from elementary torch operations in 32 bits (``own`` false) or through
``bit_gemv_i2_amd`` (``own`` true).  ``exact`` is the definition in 64 bits.

Weights are ternary, T int8 [N][K] with a scale for each row and 128 columns, S fp32 [N][K/128]; activations are int8 codes
[M][K] with a factor for each token.  ``prepare`` holds the weights both ways, as these and in the library's tile layout.
The norm's codes are defined in fp32, operation by operation behind a mean square in 64 bits, so that they are compared as
the whole numbers that they are.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = float(np.float32(1e-5))
ACTS = ("none", "relu", "relu2", "silu", "gelu")
MOST_NORM = 16383 * 2560           # values of the largest listed norm
MOST_WEIGHTS = 20480 * 3200        # the widest product of the framework's benchmark
MOST_EXPERTS = 64 * 2560 * 1280    # weights of the most experts listed
MOST_PRODUCT = 8190 * 6912 * 2560  # multiplications of the largest listed product
MOST_ROUTED = 16383 * 128          # logits of the largest listed routing


def _norm(name, M, K, dtype, add, parts=0):
    return {"name": name, "op": "norm", "M": M, "K": K, "dtype": dtype, "add": add, "parts": parts}


def _linear(name, M, N, K, act, gated, bias, residual, out):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "act": act, "gated": gated, "bias": bias,
            "residual": residual, "out": out}


def _grouped(name, T, k, E, N, K, act, gated, bias, gather, out):
    return {"name": name, "op": "grouped", "T": T, "k": k, "E": E, "N": N, "K": K, "act": act, "gated": gated, "bias": bias,
            "gather": gather, "out": out}


def _route(name, T, E, k, padded, dtype):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "padded": padded, "dtype": dtype}


def listed():
    return [
        # one user's token between two products of the 2560-wide model
        _norm("norm_1x2560", 1, 2560, "float32", "float32"),
        # a prefill of 512 tokens, each with what six experts gave
        _norm("norm_512_of_6_experts", 512, 2560, "float32", "bfloat16", 6),
        # a packed prefill of an odd number of tokens
        _norm("norm_16383x2560", 16383, 2560, "bfloat16", "bfloat16"),
        # the down projection of one token, added to the residual stream
        _linear("linear_1x2560x6912", 1, 2560, 6912, "none", False, False, "float32", "float32"),
        # gate and up projections of 8 users' tokens, squared ReLU
        _linear("linear_8x13824x2560", 8, 13824, 2560, "relu2", True, False, None, "bfloat16"),
        # the same for the 512-token prefill
        _linear("linear_512x13824x2560", 512, 13824, 2560, "relu2", True, False, None, "bfloat16"),
        # the output projection of a packed prefill with a bias, added to the residual stream
        _linear("linear_4001x2560x2560", 4001, 2560, 2560, "none", False, True, "bfloat16", "bfloat16"),
        # one token, two of eight experts, gate and up projections
        _grouped("grouped_1_to_2_of_8", 1, 2, 8, 6912, 2560, "silu", True, False, True, "bfloat16"),
        # 24 users' tokens, six of 64 small experts each, down projections
        _grouped("grouped_24_to_6_of_64", 24, 6, 64, 2560, 1280, "none", False, False, False, "float32"),
        # a packed prefill, two of eight experts, gate and up projections
        _grouped("grouped_4095_to_2_of_8", 4095, 2, 8, 6912, 2560, "relu2", True, False, True, "bfloat16"),
        # the router of a serving step of 16 users, two places of them empty
        _route("route_16_to_6_of_64", 16, 64, 6, 2, "float32"),
        # the router of a packed prefill, its last rows padding
        _route("route_16383_to_8_of_128", 16383, 128, 8, 100, "bfloat16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "grouped", "route"))
    dtype = rng.choice(("bfloat16", "float32"))
    other = rng.choice(("bfloat16", "float32"))
    K = 128 * _log(rng, 1, 64)
    N = 32 * _log(rng, 1, 640)
    act = rng.choice(ACTS)
    gated = rng.random() < 0.5
    bias = rng.random() < 0.4
    if op == "norm":
        K = 16 * _log(rng, 2, 1024)
        parts = rng.choice((0, 0, 1, 2, 6, 8))
        M = _log(rng, 1, max(1, min(16383, MOST_NORM // (K * max(1, parts)))))
        c = _norm("", M, K, dtype, other if parts else rng.choice((None, other, other)), parts)
    elif op == "linear":
        N = min(N, MOST_WEIGHTS // K // 32 * 32)
        M = _log(rng, 1, max(1, min(8192, MOST_PRODUCT // (N * K))))
        c = _linear("", M, N, K, act, gated, bias, rng.choice((None, "bfloat16", "float32")), dtype)
    elif op == "grouped":
        E = rng.choice((4, 8, 16, 32, 64))
        k = rng.randint(1, min(8, E))
        N = max(32, min(N, MOST_EXPERTS // (E * K) // 32 * 32))
        T = _log(rng, 1, max(1, min(4096, MOST_PRODUCT // (N * K * k))))
        c = _grouped("", T, k, E, N, K, act, gated, bias, rng.random() < 0.5, dtype)
    else:
        E = rng.choice((4, 8, 16, 60, 64, 128, 256))
        T = _log(rng, 1, min(16383, MOST_ROUTED // E))
        c = _route("", T, E, rng.randint(1, min(8, E)), rng.randint(0, T - 1) if rng.random() < 0.4 else 0, dtype)
    del c["name"]
    return c


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(g, *shape):
    """int8 codes as the quantiser leaves them: bell-shaped, the largest near 127."""
    return torch.clamp(torch.round(_normal(g, *shape) * 36.0), -127, 127).to(torch.int8)


def _weights(g, N, K):
    """Ternary weights whose product keeps the size of its input, and their scales."""
    T = torch.randint(-1, 2, (N, K), generator=g, device="cuda", dtype=torch.int8)
    return T, (0.5 + _uniform(g, N, K // 128)) / math.sqrt(K * 2 / 3)


def _tiles(T, S):
    """The library's layout: bricks of 16 rows x 128 columns, 2-bit codes of 4 columns four apart in a byte; scales 16 rows a block."""
    N, K = T.shape
    c = (T & 3).view(torch.uint8).view(N // 16, 16, K // 128, 2, 4, 4, 4)  # row, block, word, lane group, field, byte
    b = c[..., 0, :] | c[..., 1, :] << 2 | c[..., 2, :] << 4 | c[..., 3, :] << 6
    packed = b.permute(0, 2, 4, 1, 3, 5).contiguous().view(-1)
    return packed, S.view(N // 16, 16, K // 128).transpose(1, 2).contiguous().view(-1)


def _chosen(case):
    """The experts of each token [T][k], fixed by the case: some are asked for more than others."""
    r = np.random.default_rng([case["T"], case["k"], case["E"], case["N"], case["K"]])
    score = r.standard_normal((case["T"], case["E"])) + 0.5 * r.standard_normal(case["E"])
    return np.argsort(-score, axis=1, kind="stable")[:, : case["k"]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": dict(case)}
    op = case["op"]
    if op == "norm":
        M, K, parts = case["M"], case["K"], case["parts"]
        # a residual stream: a few wide channels, tokens of different sizes
        s["x"] = (_normal(g, M, K) * torch.exp(0.5 * _normal(g, 1, K)) * torch.exp(0.3 * _normal(g, M, 1))).to(getattr(torch, case["dtype"]))
        s["weight"] = 1.0 + 0.1 * _normal(g, K)
        s["add"] = s["slots"] = s["gates"] = None
        if case["add"]:
            s["add"] = (_normal(g, M * max(1, parts), K) * 0.5).to(getattr(torch, case["add"]))
        if parts:
            s["slots"] = torch.randperm(M * parts, generator=g, device="cuda").to(torch.int32).view(M, parts)
            s["slots"].masked_fill_(_uniform(g, M, parts) < 0.02, -1)  # a place that no expert took
            s["gates"] = torch.softmax(_normal(g, M, parts), -1)
        return s
    if op == "route":
        T, E = case["T"], case["E"]
        s["logits"] = (_normal(g, T, E) * 1.5 + 0.5 * _normal(g, 1, E)).to(getattr(torch, case["dtype"]))
        if case["padded"]:
            s["logits"][T - case["padded"]:] = -math.inf
        return s
    N, K = case["N"], case["K"]
    groups = case["E"] if op == "grouped" else 1
    s["T"], s["S"] = _weights(g, groups * N, K)
    s["packed"], s["scales"] = _tiles(s["T"], s["S"])
    s["bias"] = None
    if case["bias"]:
        s["bias"] = 0.3 * _normal(g, groups, N) if op == "grouped" else 0.3 * _normal(g, N)
    M = case["M"] if op == "linear" else case["T"]
    rows = M
    if op == "grouped":
        chosen = torch.from_numpy(_chosen(case)).cuda()[torch.randperm(M, generator=g, device="cuda")].flatten()
        order = torch.argsort(chosen, stable=True)
        s["rows"] = (order // case["k"]).to(torch.int32) if case["gather"] else None
        s["starts"] = _before(torch.bincount(chosen, minlength=groups))
        rows = M * case["k"]
    tokens = M if op == "linear" or case["gather"] else rows
    s["q"] = _codes(g, tokens, K)
    s["s_a"] = torch.exp(0.3 * _normal(g, tokens)) / 36.0
    s["residual"] = None
    if op == "linear" and case["residual"]:
        s["residual"] = _normal(g, M, N // 2 if case["gated"] else N).to(getattr(torch, case["residual"]))
    return s


def _before(counts):
    """int32 [n + 1]: how many stand before each, and in all."""
    return torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)


def work(case):
    size = {"float32": 4, "bfloat16": 2, None: 0}
    op = case["op"]
    if op == "norm":
        M, K, P = case["M"], case["K"], case["parts"]
        x, add = size[case["dtype"]], size[case["add"]]
        each = x + (x + add * max(1, P) if add else 0) + 1
        return {"bytes": M * K * each + 4 * K + M * (4 + 8 * P), "flops": M * K * (6 + (2 * P if P else bool(add)))}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * size[case["dtype"]] + T * k * 16 + 4 * E + 4, "flops": T * E}
    N, K = case["N"], case["K"]
    wide = N // 2 if case["gated"] else N
    weights = N * K // 4 + N * K // 32 + (4 * N if case["bias"] else 0)
    if op == "linear":
        rows = tokens = case["M"]
    else:
        rows = case["T"] * case["k"]
        tokens = case["T"] if case["gather"] else rows
        weights *= len(np.unique(_chosen(case)))
    out = wide * (size[case["out"]] + size[case.get("residual")])
    return {"bytes": weights + tokens * (K + 4) + rows * (out + (4 if op == "grouped" and case["gather"] else 0)), "flops": 2 * rows * N * K}


# ------------------------------------------------------------------ the plain forms
def _divide(a, b):
    """a / b with b as a tensor: division by a Python number may be a product with its rounded inverse."""
    return a / torch.full_like(a, b)


def _norm_plain(s):
    x, add = s["x"], s["add"]
    if s["slots"] is not None:
        d = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        for j in range(s["slots"].shape[1]):
            slot = s["slots"][:, j].long()
            part = s["gates"][:, j, None] * add[slot.clamp(min=0)].float()
            d = torch.where((slot >= 0)[:, None], d + part, d)
        x = (x.float() + d).to(x.dtype)
    elif add is not None:
        x = (x.float() + add.float()).to(x.dtype)
    v = x.float()
    mean = v.double().square().sum(-1) / v.shape[1]  # 64 bits: a code next to a rounding border follows the last bit
    r = (1.0 / torch.sqrt(mean + EPS)).float()
    h = (v * r[:, None]) * s["weight"]
    most = h.abs().amax(-1).clamp(min=1e-5)
    inv = torch.full_like(most, 127.0) / most
    codes = torch.clamp(torch.round(h * inv[:, None]), -127, 127).to(torch.int8)
    return {"codes": codes, "s_a": _divide(most, 127.0), "x": x}


def _act(z, act, gated):
    if gated:
        z, up = z[:, : z.shape[1] // 2], z[:, z.shape[1] // 2:]
    if act == "relu":
        z = torch.clamp(z, min=0.0)
    elif act == "relu2":
        z = torch.clamp(z, min=0.0).square()
    elif act == "silu":
        z = z / (1.0 + torch.exp(-z))
    elif act == "gelu":
        z = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z * up if gated else z


def _dense(T, S):
    """Ternary weights with their scales, fp32 [K][N]."""
    return (T.float().unflatten(1, (-1, 128)) * S[:, :, None]).flatten(1).t()


def _linear_plain(s):
    case = s["case"]
    z = (s["q"].float() @ _dense(s["T"], s["S"])) * s["s_a"][:, None]
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, case["act"], case["gated"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(getattr(torch, case["out"]))


def _grouped_plain(s):
    case, N = s["case"], s["case"]["N"]
    starts = s["starts"].tolist()  # a program of plain operations has to know how many rows each expert has
    y = torch.empty((starts[-1], N // 2 if case["gated"] else N), dtype=getattr(torch, case["out"]), device="cuda")
    for e, (lo, hi) in enumerate(zip(starts, starts[1:])):
        if lo == hi:
            continue
        at = s["rows"][lo:hi].long() if case["gather"] else slice(lo, hi)
        W = _dense(s["T"][e * N: (e + 1) * N], s["S"][e * N: (e + 1) * N])
        z = (s["q"][at].float() @ W) * s["s_a"][at][:, None]
        if s["bias"] is not None:
            z = z + s["bias"][e]
        y[lo:hi] = _act(z, case["act"], case["gated"]).to(y.dtype)
    return y


def _route_plain(s):
    case, logits = s["case"], s["logits"].float()
    T, E, k = case["T"], case["E"], case["k"]
    value, chosen = torch.sort(logits, dim=1, descending=True, stable=True)
    value, chosen = value[:, :k], chosen[:, :k]
    there = value > -math.inf
    gates = torch.exp(value - value[:, :1].clamp(min=-3e38)) * there
    gates = gates / gates.sum(-1, keepdim=True).clamp(min=1e-30)
    chosen = torch.where(there, chosen, torch.full_like(chosen, E))  # those that chose none stand behind the last expert
    order = torch.argsort(chosen.flatten(), stable=True)
    starts = _before(torch.bincount(chosen.flatten(), minlength=E + 1)[:E])
    place = torch.arange(T * k, device="cuda")
    slots = torch.empty_like(order).index_put_((order,), place)
    rows = torch.where(place < starts[E], order // k, torch.full_like(order, -1))
    whole = torch.int32
    return {"experts": torch.where(there, chosen, torch.full_like(chosen, -1)).to(whole), "gates": gates, "starts": starts,
            "rows": rows.to(whole), "slots": torch.where(there, slots.view(T, k), torch.full_like(chosen, -1)).to(whole)}


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"norm": _norm_plain, "linear": _linear_plain, "grouped": _grouped_plain, "route": _route_plain}[op](s)
    import bit_gemv_i2_amd as bn
    if op == "norm":
        q, s_a, x = bn.bitnet_add_norm_quant(s["x"], s["weight"], EPS, add=s["add"], slots=s["slots"], gates=s["gates"])
        return {"codes": q, "s_a": s_a, "x": x}
    if op == "route":
        experts, gates, starts, rows, slots = bn.bitnet_route(s["logits"], case["k"])
        return {"experts": experts, "gates": gates, "starts": starts, "rows": rows, "slots": slots}
    out = getattr(torch, case["out"])
    if op == "linear":
        return bn.bitnet_w2a8_linear(s["packed"], s["scales"], s["q"], s["s_a"], case["N"], case["K"], bias=s["bias"],
                                     act=case["act"], gated=case["gated"], residual=s["residual"], out_dtype=out)
    return bn.bitnet_w2a8_grouped(s["packed"], s["scales"], s["q"], s["s_a"], s["starts"], case["N"], case["K"], rows=s["rows"],
                                  bias=s["bias"], act=case["act"], gated=case["gated"], out_dtype=out)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_norm(s):
    v = s["x"].double()
    if s["gates"] is not None:
        padded = torch.cat([s["add"].double(), s["add"].new_zeros(1, v.shape[1]).double()])  # slot -1 is the row of zeros
        for j in range(s["slots"].shape[1]):
            v = v + s["gates"][:, j, None].double() * padded[s["slots"][:, j].long()]
    elif s["add"] is not None:
        v = v + s["add"].double()
    seen = v.to(s["x"].dtype).double()  # the norm is of the stored stream
    h = seen * torch.rsqrt(seen.pow(2).mean(-1, keepdim=True) + EPS) * s["weight"].double()
    return {"codes": None, "s_a": torch.clamp(h.abs().amax(-1), min=1e-5) / 127, "x": v}


def _exact_product(T, S, q, s_a, bias, act, gated):
    """Whole block sums, each with its scale, in float64; then the activation."""
    z = torch.zeros((q.shape[0], T.shape[0]), dtype=torch.float64, device=q.device)
    for b in range(S.shape[1]):
        z += (q[:, 128 * b: 128 * (b + 1)].double() @ T[:, 128 * b: 128 * (b + 1)].double().t()) * S[:, b].double()
    z = z * s_a.double()[:, None]
    if bias is not None:
        z = z + bias.double()
    up = None
    if gated:
        z, up = z.chunk(2, dim=1)
    if act == "relu":
        z = z.relu()
    elif act == "relu2":
        z = z.relu() ** 2
    elif act == "silu":
        z = z * z.sigmoid()
    elif act == "gelu":
        z = z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z if up is None else z * up


def _exact_linear(s):
    case = s["case"]
    y = _exact_product(s["T"], s["S"], s["q"], s["s_a"], s["bias"], case["act"], case["gated"])
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_grouped(s):
    case, N = s["case"], s["case"]["N"]
    T, S = s["T"].view(-1, N, case["K"]), s["S"].view(case["E"], N, -1)
    q, s_a = (s["q"][s["rows"].long()], s["s_a"][s["rows"].long()]) if case["gather"] else (s["q"], s["s_a"])
    counts = torch.diff(s["starts"]).tolist()
    parts = [_exact_product(T[e], S[e], qe, se, None if s["bias"] is None else s["bias"][e], case["act"], case["gated"])
             for e, (qe, se) in enumerate(zip(q.split(counts), s_a.split(counts)))]
    return torch.cat(parts)


def _exact_route(s):
    logits = s["logits"].double().cpu().numpy()
    T, E = logits.shape
    k = s["case"]["k"]
    experts = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    value = np.take_along_axis(logits, experts, 1)
    gates = np.where(np.isfinite(value), np.exp(value - np.maximum(value[:, :1], -1e300)), 0.0)
    gates /= np.maximum(gates.sum(1, keepdims=True), 1e-300)
    experts = np.where(np.isfinite(value), experts, -1).astype(np.int32)
    rows, starts = np.full(T * k, -1, np.int32), [0]
    slots = np.full((T, k), -1, np.int32)
    for e in range(E):
        token, place = np.nonzero(experts == e)
        at = starts[-1] + np.arange(len(token))
        rows[at], slots[token, place] = token, at
        starts.append(starts[-1] + len(token))
    return {"experts": experts, "gates": gates, "starts": np.array(starts, np.int32), "rows": rows, "slots": slots}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "grouped": _exact_grouped, "route": _exact_route}[case["op"]](s)
