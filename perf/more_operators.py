"""What the unit's products are measured on: the cases, their inputs, their plain
form in elementary torch operations, and their values in 64 bits.

Three operators around one FSDP unit (R virtual ranks; parameters in full-unit
order, shards in buffers [R][S], as everywhere in this package):

  gather8   the all-gather of a unit with its matrices in 8 bits: for every row
            (along a parameter's last dimension) of largest magnitude a, the
            scale s = a / 127 and the codes c = round(x 127 / a); each receiver
            reads its unit back as c s, other parameters as they are
  linear8   a linear layer on such codes.  forward: tokens quantised row by row
            like the weights, Y = (Cx Cw^T) sx sw.  input gradient: dY times
            the weights' channel scales, quantised row by row, dX = (Cd Cw) sd
  grouped   linear layers of experts, rows of tokens sorted by expert.
            forward: Y[rows of g] = X[rows of g] W_g^T.  gradients: dX[rows of
            g] = dY[rows of g] W_g and dW_g = dY[rows of g]^T X[rows of g]

Weights are [out, in], of experts [groups, out, in].
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK_512 = "512x512,512x512,512x512,512x512,512x2048,2048x512,512,512"
BLOCK_4096 = ("4096x4096,1024x4096,1024x4096,4096x4096,14336x4096,4096x14336,14336x4096,"
              "4096,4096")


def listed():
    return [
        # one transformer block of hidden 512 over four ranks: the smallest unit a
        # step gathers, where latency counts
        {"name": "gather8-block512-r4", "op": "gather8", "shapes": BLOCK_512, "R": 4,
         "layout": "per_param", "type": "bf16"},
        # a block of hidden 4096 over eight ranks: 218M parameters, bound by memory
        {"name": "gather8-block4096-flat-r8", "op": "gather8", "shapes": BLOCK_4096, "R": 8,
         "layout": "flat", "type": "bf16"},
        # a single token through the hidden-4096 block's up projection: 59 MB of
        # codes are read for it, latency and memory
        {"name": "linear8-1x14336x4096", "op": "linear8", "dir": "forward", "rows": 1,
         "groups": 1, "out": 14336, "in": 4096},
        # a micro-batch of 2048 tokens through the hidden-512 block's
        {"name": "linear8-2048x2048x512", "op": "linear8", "dir": "forward", "rows": 2048,
         "groups": 1, "out": 2048, "in": 512},
        # 8192 tokens through the hidden-4096 block's: bound by the matrix cores
        {"name": "linear8-8192x14336x4096", "op": "linear8", "dir": "forward", "rows": 8192,
         "groups": 1, "out": 14336, "in": 4096},
        # odd sizes, three experts, backward: rows of codes end inside a load
        {"name": "linear8-grad-777x1025x2049-g3", "op": "linear8", "dir": "input_grad",
         "rows": 777, "groups": 3, "out": 1025, "in": 2049},
        # the input gradient of the hidden-4096 block's down projection
        {"name": "linear8-grad-8192x4096x14336", "op": "linear8", "dir": "input_grad",
         "rows": 8192, "groups": 1, "out": 4096, "in": 14336},
        # a few tokens, one expert without any: every other expert's weights are
        # read for two or three rows each
        {"name": "grouped-16x2048x512-g8", "op": "grouped", "dir": "forward", "rows": 16,
         "tail": 0, "groups": 8, "out": 2048, "in": 512, "type": "bf16", "grad": "bf16"},
        # training in fp32, odd sizes, rows behind the last expert's
        {"name": "grouped-1000x333x510-g5-f32", "op": "grouped", "dir": "forward",
         "rows": 1000, "tail": 24, "groups": 5, "out": 333, "in": 510, "type": "f32",
         "grad": "f32"},
        # 16384 tokens over eight experts of the hidden-4096 block's size
        {"name": "grouped-16384x14336x4096-g8", "op": "grouped", "dir": "forward",
         "rows": 16384, "tail": 0, "groups": 8, "out": 14336, "in": 4096, "type": "bf16",
         "grad": "bf16"},
        # the backward pass of sixteen small experts, weight gradients added to
        # fp32 accumulators over micro-batches
        {"name": "grouped-grads-8192x2048x512-g16", "op": "grouped", "dir": "grads",
         "rows": 8192, "tail": 0, "groups": 16, "out": 2048, "in": 512, "type": "bf16",
         "grad": "f32"},
        # and of the eight large ones, gradients in bf16 as the replicas are
        {"name": "grouped-grads-16384x14336x4096-g8", "op": "grouped", "dir": "grads",
         "rows": 16384, "tail": 0, "groups": 8, "out": 14336, "in": 4096, "type": "bf16",
         "grad": "bf16"},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["gather8", "linear8", "linear8", "grouped", "grouped"])
    if op == "gather8":
        shapes = [(size(1, 4096), size(1, 4096))]
        for _ in range(rng.randint(0, 7)):
            kind = rng.random()
            if kind < 0.2:
                shapes.append((size(1, 4096),))                              # a scale or a bias
            elif kind < 0.35:
                shapes.append((size(1, 16), size(1, 1024), size(1, 1024)))   # experts
            else:
                shapes.append((size(1, 4096), size(1, 4096)))
        return {"op": op, "shapes": ",".join("x".join(map(str, s)) for s in shapes),
                "R": rng.choice([1, 2, 3, 4, 5, 8]), "layout": rng.choice(["per_param", "flat"]),
                "type": rng.choice(["bf16", "bf16", "f32"])}

    def side():
        n = size(32, 8192)
        return n if rng.random() < 0.3 else -(-n // 64) * 64

    case = {"op": op, "rows": size(1, 16384), "groups": rng.choice([1, 1, 2, 3, 5, 8, 16, 32]),
            "out": side(), "in": side()}
    while case["groups"] > 1 and case["groups"] * case["out"] * case["in"] > 2 ** 28:
        case["groups"] //= 2
    while case["rows"] * case["out"] * case["in"] > 2 ** 38:
        case["rows"] //= 2
    if op == "linear8":
        case["dir"] = rng.choice(["forward", "input_grad"])
        return case
    case["dir"] = rng.choice(["forward", "grads"])
    case["tail"] = rng.choice([0, 0, 3, 50])
    case["type"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
    case["grad"] = "f32" if case["type"] == "f32" else rng.choice(["bf16", "f32"])
    if case["type"] == "f32":        # costs sixteen times as much
        case["rows"] = min(case["rows"], 2048)
    return case


# ------------------------------------------------------------------- layout
def shapes_of(case):
    return [tuple(int(d) for d in s.split("x")) for s in case["shapes"].split(",")]


def places(case):
    """(parameter, offset in the unit, shape) of every parameter."""
    shapes = shapes_of(case)
    numel = [math.prod(s) for s in shapes]
    return [(p, sum(numel[:p]), s) for p, s in enumerate(shapes)]


def total(case):
    return sum(math.prod(s) for s in shapes_of(case))


def shard_size(case):
    if case["layout"] == "flat":
        return -(-total(case) // case["R"])
    return sum(-(-s[0] // case["R"]) * (math.prod(s) // s[0]) for s in shapes_of(case))


def take_full(case, shards):
    """The parameters' values out of a buffer [R][S], each in its shape: views of
    it where the layout has them whole."""
    R, S = case["R"], shard_size(case)
    if case["layout"] == "flat":
        return [shards[at:at + math.prod(s)].view(s) for _, at, s in places(case)]
    row = [math.prod(s) // s[0] for s in shapes_of(case)]
    k = [-(-s[0] // R) for s in shapes_of(case)]
    begin = [sum(x * y for x, y in zip(k[:p], row[:p])) for p in range(len(k))]
    return [shards.view(R, S)[:, begin[p]:begin[p] + k[p] * row[p]].reshape(
        R * k[p], row[p])[:s[0]].reshape(s) for p, _, s in places(case)]


def sizes_of(case):
    """Rows of every group, as a router leaves them: from many to few, the last of
    four or more without any."""
    n, E = case["rows"], case["groups"]
    share = [1.0 / (g + 3) for g in range(E)]
    if E >= 4:
        share[-1] = 0.0
    ends = [int(round(n * sum(share[:g + 1]) / sum(share))) for g in range(E)]
    sizes = [b - a for a, b in zip([0] + ends, ends)]
    return sizes[1::2] + sizes[0::2]


def pitch(k):
    """Bytes from one row of codes to the next."""
    return -(-k // 16) * 16


# ------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uneven(rows, cols):
        """Activations and their gradients: rows of different sizes, a few
        channels much larger than the others."""
        x = normal(rows, cols) * torch.exp(0.5 * normal(rows, 1))
        return x * torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 8.0, 1.0)

    if case["op"] == "gather8":
        full = normal(case["R"] * shard_size(case)).mul_(0.02)
        state["shards"] = full.to(TYPES[case["type"]])
        if own:
            import fully_sharded_amd as F
            # what a training program keeps per unit: the plan, the choice of the
            # matrices that travel in 8 bits, every rank's receive buffers, and
            # the calls bound to them
            plan = F.Plan(shapes_of(case), case["R"], case["layout"])
            qu = F.Quant(plan)
            qu.prepare()
            codes, scales, rest, units = [], [], [], []
            [(codes.append(qu.code_buffer()), scales.append(qu.scale_buffer()),
              rest.append(qu.rest_buffer(TYPES[case["type"]])),
              units.append(torch.empty(plan.T, dtype=TYPES[case["type"]], device="cuda")))
             for _ in range(case["R"])]
            state["gather"] = F.bind_gather_quantize(qu, state["shards"], codes, scales, rest)
            state["read"] = F.bind_dequantize(qu, codes, scales, rest, units)
            state["units"] = units
        return state

    E, n, k = case["groups"], case["out"], case["in"]
    state["sizes"] = sizes_of(case)
    state["offsets"] = torch.tensor([sum(state["sizes"][:i]) for i in range(E + 1)],
                                    dtype=torch.int32, device="cuda")
    w = torch.randn(E, n, k, generator=g, device="cuda", dtype=torch.bfloat16) / math.sqrt(k)
    if case["op"] == "linear8":
        # the codes as a quantised gather leaves them, rows padded to 16 bytes
        c, s = quantize(w.float())
        state["codes"] = torch.zeros(E, n, pitch(k), dtype=torch.int8, device="cuda")
        state["codes"][:, :, :k] = c.to(torch.int8)
        state["codes"] = state["codes"][:, :, :k]
        state["scales"] = s.view(E, n)
        cols, outs = (k, n) if case["dir"] == "forward" else (n, k)
        state["x"] = uneven(case["rows"], cols).bfloat16()
        state["y"] = torch.zeros(case["rows"], outs, dtype=torch.bfloat16, device="cuda")
        if own:
            import fully_sharded_amd as F
            xq = torch.empty(case["rows"], pitch(cols), dtype=torch.int8,
                             device="cuda")[:, :cols]
            sx = torch.empty(case["rows"], device="cuda")
            ends = None if E == 1 else state["offsets"]
            if case["dir"] == "forward":
                state["quantize"] = F.bind_quantize_rows(state["x"], xq, sx)
                state["product"] = F.bind_grouped_matmul_i8(
                    "nt", xq, sx, state["codes"], state["scales"], state["y"], offsets=ends)
            else:
                state["quantize"] = F.bind_quantize_rows(state["x"], xq, sx,
                                                         channel=state["scales"], offsets=ends)
                state["product"] = F.bind_grouped_matmul_i8(
                    "nn", xq, sx, state["codes"], None, state["y"], offsets=ends)
        return state

    dt, rows = TYPES[case["type"]], case["rows"] + case["tail"]
    state["w"] = w.to(dt)
    state["x"] = uneven(rows, k).to(dt)
    if case["dir"] == "forward":
        state["y"] = normal(rows, n).to(dt)
    else:
        state["dy"] = (1e-3 * uneven(rows, n)).to(dt)
        state["dx"] = (1e-3 * normal(rows, k)).to(dt)
        state["dw"] = (1e-3 * normal(E, n, k)).to(TYPES[case["grad"]])
    if own:
        import fully_sharded_amd as F
        add = case["dir"] == "grads" and case["type"] != case["grad"]
        if case["dir"] == "forward":
            state["calls"] = [F.bind_grouped_matmul("nt", state["x"], state["w"], state["y"],
                                                    offsets=state["offsets"])]
        else:
            state["calls"] = [
                F.bind_grouped_matmul("nn", state["dy"], state["w"], state["dx"],
                                      offsets=state["offsets"]),
                F.bind_grouped_matmul("tn", state["dy"], state["x"], state["dw"],
                                      offsets=state["offsets"], accumulate=add)]
    return state


# --------------------------------------------------------------------- runs
def quantize(x):
    """Codes (whole numbers in fp32) and scales [..., 1] of the rows of an fp32 x."""
    a = x.abs().amax(-1, keepdim=True)
    return torch.round(x * (127.0 / a)), a / 127.0


def plain(state):
    case = state["case"]
    if case["op"] == "gather8":
        dt = TYPES[case["type"]]

        def read_back(v):
            if v.dim() < 2:
                return v.reshape(-1)
            c, s = quantize(v.float())
            return (c * s).to(dt).reshape(-1)

        unit = torch.cat([read_back(v) for v in take_full(case, state["shards"])])
        return [unit.clone() for _ in range(case["R"])]
    sizes = state["sizes"]
    used = sum(sizes)
    if case["op"] == "linear8":
        x, w = state["x"].float().split(sizes), state["codes"].float()
        if case["dir"] == "forward":
            q = [quantize(xg) for xg in x]
            state["y"].copy_(torch.cat([(c @ wg.T) * s * t for (c, s), wg, t in
                                        zip(q, w, state["scales"])]))
        else:
            q = [quantize(xg * t) for xg, t in zip(x, state["scales"])]
            state["y"].copy_(torch.cat([(c @ wg) * s for (c, s), wg in zip(q, w)]))
        return {"y": state["y"]}
    w, x = state["w"].float(), state["x"][:used].float().split(sizes)
    if case["dir"] == "forward":
        state["y"][:used].copy_(torch.cat([xg @ wg.T for xg, wg in zip(x, w)]))
        return {"y": state["y"]}
    dy = state["dy"][:used].float().split(sizes)
    state["dx"][:used].copy_(torch.cat([dg @ wg for dg, wg in zip(dy, w)]))
    dw = torch.stack([dg.T @ xg for dg, xg in zip(dy, x)])
    state["dw"].copy_(dw if case["type"] == case["grad"] else state["dw"] + dw)
    return {"dx": state["dx"], "dw": state["dw"]}


def run(state):
    if not own:
        return plain(state)
    case = state["case"]
    if case["op"] == "gather8":
        state["gather"]()
        state["read"]()
        return state["units"]
    if case["op"] == "linear8":
        state["quantize"]()
        state["product"]()
        return {"y": state["y"]}
    [call() for call in state["calls"]]
    if case["dir"] == "forward":
        return {"y": state["y"]}
    return {"dx": state["dx"], "dw": state["dw"]}


# --------------------------------------------------------------------- work
def work(case):
    es = {"bf16": 2, "f32": 4}
    if case["op"] == "gather8":
        # the shards once; per rank the codes and scales written and read, and
        # the unit written
        m = [math.prod(s) for s in shapes_of(case) if len(s) > 1]
        rows = sum(math.prod(s[:-1]) for s in shapes_of(case) if len(s) > 1)
        T, R, e = total(case), case["R"], es[case["type"]]
        other = T - sum(m)
        return {"bytes": T * e + R * (2 * (sum(m) + 4 * rows) + 2 * other * e + T * e),
                "flops": (3 + R) * T}
    n, k, rows = case["out"], case["in"], case["rows"]
    met = sum(s > 0 for s in sizes_of(case))     # groups that have rows
    if case["op"] == "linear8":
        a, c = (k, n) if case["dir"] == "forward" else (n, k)
        return {"bytes": rows * (2 * a + 2 * c) + met * n * (k + 4), "flops": 2 * rows * n * k}
    e, ge = es[case["type"]], es[case["grad"]]
    if case["dir"] == "forward":
        return {"bytes": rows * (k + n) * e + met * n * k * e, "flops": 2 * rows * n * k}
    old = (met if ge != e else 0) * n * k * ge   # what the gradients are added to
    new = (met if ge != e else case["groups"]) * n * k * ge
    return {"bytes": rows * (2 * k + n) * e + met * n * k * e + old + new,
            "flops": 4 * rows * n * k}


# ------------------------------------------------------------ in 64 bits
def shard_index(case):
    """For every element of the unit, its place in the buffer [R][S]."""
    R, S, T = case["R"], shard_size(case), total(case)
    if case["layout"] == "flat":
        i = torch.arange(T, device="cuda")
        return i // S * S + i % S
    parts, at = [], 0
    for s in shapes_of(case):
        row = math.prod(s) // s[0]
        k = -(-s[0] // R)
        i = torch.arange(s[0], device="cuda")
        parts.append(((i // k * S + at + i % k * row)[:, None] +
                      torch.arange(row, device="cuda")[None]).view(-1))
        at += k * row
    return torch.cat(parts)


def exact_codes(x):
    """What a row's codes stand for, in units of its scale, and the scale."""
    a = x.abs().max(dim=1, keepdim=True).values
    return torch.round(127 * x / a), a / 127


def exact(case, seed):
    global own
    kept, own = own, False
    state = prepare(case, seed)
    own = kept
    if case["op"] == "gather8":
        index, out = shard_index(case), None
        out = torch.empty(total(case), dtype=torch.float64, device="cuda")
        for _, at, s in places(case):
            n = math.prod(s)
            v = state["shards"][index[at:at + n]].double()
            if len(s) > 1:
                c, scale = exact_codes(v.view(-1, s[-1]))
                v = (c * scale).view(-1)
            out[at:at + n] = v
        return [out] * case["R"]
    ends = state["offsets"].tolist()
    if case["op"] == "linear8":
        y = torch.zeros(state["y"].shape, dtype=torch.float64, device="cuda")
        for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if lo == hi:
                continue
            x, w = state["x"][lo:hi].double(), state["codes"][g].double()
            t = state["scales"][g].double()
            if case["dir"] == "forward":
                c, s = exact_codes(x)
                y[lo:hi] = torch.einsum("tk,nk->tn", c, w) * s * t[None, :]
            else:
                c, s = exact_codes(x * t[None, :])
                y[lo:hi] = torch.einsum("tn,nk->tk", c, w) * s
        return {"y": y}
    if case["dir"] == "forward":
        y = state["y"].double()
        for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
            y[lo:hi] = torch.einsum("tk,nk->tn", state["x"][lo:hi].double(),
                                    state["w"][g].double())
        return {"y": y}
    dx, dw = state["dx"].double(), state["dw"].double()
    if case["type"] == case["grad"]:
        dw.zero_()
    for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
        d, x = state["dy"][lo:hi].double(), state["x"][lo:hi].double()
        dx[lo:hi] = torch.einsum("tn,nk->tk", d, state["w"][g].double())
        dw[g] += torch.einsum("tn,tk->nk", d, x)
    return {"dx": dx, "dw": dw}
