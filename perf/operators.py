"""What the Muon operators are measured on: the cases, their inputs, their plain
form in elementary torch operations, and their values in 64 bits.

Three operators, in the order in which a sharded training step runs them over
one FSDP unit (R virtual ranks; parameters in full-unit order in buffers of T
elements, shards in buffers [R][S], as everywhere in this package):

  momentum       mean of the R gradient replicas, the momentum's shards
                 m <- mu m + (1 - mu) g, and the gathered update
                 u = (1 - mu) g + mu m (Nesterov) or u = m
  orthogonalize  for every matrix of the unit, X = u / (|u|_F + eps), then
                 `steps` times X <- a X + (b A + c A A) X with A = X X^T
                 (of the transposed matrix where it has more rows than
                 columns)
  apply          master <- master (1 - lr wd) - lr scale X, and the
                 parameter's recast

Matrices are the parameters of two dimensions or more (the first against all
others); one-dimensional parameters are left as they are.
"""

import math

import torch

own = False

HP = {"lr": 1e-3, "momentum": 0.95, "weight_decay": 0.01, "eps": 1e-7,
      "coefficients": (3.4445, -4.7750, 2.0315), "steps": 5, "nesterov": True, "scale": "rms"}

BLOCK_512 = "512x512,512x512,512x512,512x512,512x2048,2048x512,512,512"
BLOCK_4096 = ("4096x4096,1024x4096,1024x4096,4096x4096,14336x4096,4096x14336,14336x4096,"
              "4096,4096")
RAGGED = "1000x333,777x510,1x640,1025x2049,300x3x3x7,33"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one transformer block of hidden 512 over four ranks: the smallest
        # unit a step runs, where latency counts
        {"name": "momentum-block512-r4", "op": "momentum", "shapes": BLOCK_512, "R": 4,
         "layout": "per_param", "grad": "bf16", "update": "bf16"},
        # accumulated fp32 gradients of odd sizes over three ranks: pieces and
        # rows begin off the vector grid
        {"name": "momentum-ragged-r3-f32", "op": "momentum", "shapes": RAGGED, "R": 3,
         "layout": "per_param", "grad": "f32", "update": "f32"},
        # a block of hidden 4096 over eight ranks: 218M parameters, 3.5 GB of
        # gradients, bound by memory
        {"name": "momentum-block4096-flat-r8", "op": "momentum", "shapes": BLOCK_4096, "R": 8,
         "layout": "flat", "grad": "bf16", "update": "bf16"},
        # one attention weight, the unit when every parameter is wrapped by
        # itself: pure latency
        {"name": "ortho-512", "op": "orthogonalize", "shapes": "512x512", "update": "bf16",
         "ortho": "bf16"},
        # the same block as above: six matrices of three shapes
        {"name": "ortho-block512", "op": "orthogonalize", "shapes": BLOCK_512, "update": "bf16",
         "ortho": "bf16"},
        # the 12-layer model as one unit: 72 matrices
        {"name": "ortho-model12", "op": "orthogonalize", "shapes": ",".join([BLOCK_512] * 12),
         "update": "bf16", "ortho": "bf16"},
        # the block of hidden 4096: seven matrices, bound by the matrix cores
        {"name": "ortho-block4096", "op": "orthogonalize", "shapes": BLOCK_4096,
         "update": "bf16", "ortho": "bf16"},
        # odd sizes: a tall and a wide one, a single row, one of few columns, a
        # filter bank of four dimensions
        {"name": "ortho-ragged", "op": "orthogonalize",
         "shapes": "1000x333,77x510,1x640,1025x129,300x3x3x7,33", "update": "bf16",
         "ortho": "bf16"},
        # training in fp32: the block's updates and results in fp32
        {"name": "ortho-block512-f32", "op": "orthogonalize", "shapes": BLOCK_512,
         "update": "f32", "ortho": "f32"},
        # the update of the three units' masters with the parameter's recast
        {"name": "apply-block512-r4", "op": "apply", "shapes": BLOCK_512, "R": 4,
         "layout": "per_param", "ortho": "bf16", "param": "bf16"},
        {"name": "apply-ragged-r3-f32", "op": "apply", "shapes": RAGGED, "R": 3,
         "layout": "per_param", "ortho": "f32", "param": "f32"},
        {"name": "apply-block4096-flat-r8", "op": "apply", "shapes": BLOCK_4096, "R": 8,
         "layout": "flat", "ortho": "bf16", "param": "bf16"},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["momentum", "orthogonalize", "orthogonalize", "apply"])
    shapes = []
    for _ in range(rng.randint(1, 8)):
        kind = rng.random()
        if kind < 0.15 and shapes:
            shapes.append((size(1, 4096),))                       # a scale or a bias
        elif kind < 0.3:
            shapes.append((size(4, 512), size(1, 256), 3, 3))     # a filter bank
        else:
            shapes.append((size(1, 4096), size(1, 4096)))
    if all(len(s) < 2 for s in shapes):
        shapes.append((size(16, 4096), size(16, 4096)))
    case = {"op": op, "shapes": ",".join("x".join(map(str, s)) for s in shapes)}
    if op == "orthogonalize":
        case["update"] = rng.choice(["bf16", "bf16", "f32"])
        case["ortho"] = case["update"] if rng.random() < 0.8 else rng.choice(["bf16", "f32"])
        return case
    case["R"] = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    case["layout"] = rng.choice(["per_param", "flat"])
    if op == "momentum":
        case["grad"] = rng.choice(["bf16", "f32"])
        case["update"] = rng.choice(["bf16", "f32"])
    else:
        case["ortho"] = rng.choice(["bf16", "f32"])
        case["param"] = rng.choice(["bf16", "f32"])
    return case


# ------------------------------------------------------------------- layout
def shapes_of(case):
    return [tuple(int(d) for d in s.split("x")) for s in case["shapes"].split(",")]


def places(case):
    """(parameter, offset in the unit, rows, columns) of every matrix."""
    out, at = [], 0
    for p, s in enumerate(shapes_of(case)):
        n = math.prod(s)
        if len(s) >= 2:
            out.append((p, at, s[0], n // s[0]))
        at += n
    return out


def total(case):
    return sum(math.prod(s) for s in shapes_of(case))


def shard_size(case):
    R = case["R"]
    if case["layout"] == "flat":
        return -(-total(case) // R)
    return sum(-(-s[0] // R) * (math.prod(s) // s[0]) for s in shapes_of(case))


def take_full(case, shards):
    """The matrices' values out of a buffer [R][S], in unit order: views of it
    where the layout has them whole."""
    R, S = case["R"], shard_size(case)
    if case["layout"] == "flat":
        return [shards[at:at + r * c].view(r, c) for _, at, r, c in places(case)]
    got, at = {}, 0
    for p, s in enumerate(shapes_of(case)):
        row, k = math.prod(s) // s[0], -(-s[0] // R)
        got[p] = shards.view(R, S)[:, at:at + k * row].reshape(R * k, row)[:s[0]]
        at += k * row
    return [got[p] for p, _, _, _ in places(case)]


def put_full(case, shards, values):
    """The reverse of take_full: values, one per matrix, into the buffer."""
    R, S = case["R"], shard_size(case)
    if case["layout"] == "flat":
        [shards[at:at + r * c].copy_(v.reshape(-1)) for (_, at, r, c), v in
         zip(places(case), values)]
        return
    where, at = {}, 0
    for p, s in enumerate(shapes_of(case)):
        row, k = math.prod(s) // s[0], -(-s[0] // R)
        where[p] = (at, k, row)
        at += k * row

    def put(p, rows, v):
        at, k, row = where[p]
        whole = rows // k
        shards.view(R, S)[:whole, at:at + k * row] = v[:whole * k].reshape(whole, k * row)
        if whole < R and rows > whole * k:
            shards.view(R, S)[whole, at:at + (rows - whole * k) * row] = v[whole * k:].reshape(-1)

    [put(p, r, v) for (p, _, r, _), v in zip(places(case), values)]


# ------------------------------------------------------------------- inputs
def gradient_like(g, rows, cols, sigma):
    """A matrix as gradients are: a few strong directions over white noise."""
    k = min(8, rows, cols)
    low = torch.randn(rows, k, generator=g, device="cuda") @ torch.randn(
        k, cols, generator=g, device="cuda")
    low *= 1.0 / math.sqrt(k)
    noise = torch.randn(rows, cols, generator=g, device="cuda")
    return (low + noise) * (sigma / math.sqrt(2.0))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, op = total(case), case["op"]
    state = {"case": case}

    def normal(n, sigma):
        return torch.randn(n, generator=g, device="cuda") * sigma

    def unit(sigma):
        full = torch.zeros(T, device="cuda")
        for _, at, r, c in places(case):
            full[at:at + r * c] = gradient_like(g, r, c, sigma).view(-1)
        return full

    if op == "momentum":
        n = case["R"] * shard_size(case)
        state["grads"] = [normal(T, 1e-3).to(TYPES[case["grad"]]) for _ in range(case["R"])]
        state["m"] = normal(n, 1e-4)
        state["update"] = torch.zeros(T, dtype=TYPES[case["update"]], device="cuda")
    elif op == "orthogonalize":
        state["update"] = unit(1e-3).to(TYPES[case["update"]])
        state["ortho"] = torch.zeros(T, dtype=TYPES[case["ortho"]], device="cuda")
    else:
        n = case["R"] * shard_size(case)
        state["ortho"] = unit(1.0 / math.sqrt(max(c for _, _, _, c in places(case)))).to(
            TYPES[case["ortho"]])
        state["master"] = normal(n, 0.02)
        state["param"] = torch.zeros(n, dtype=TYPES[case["param"]], device="cuda")
    if own:
        import fully_sharded_amd as F
        # the unit's plan, the choice of its matrices, the workspace and the
        # call bound to the buffers: what a training program keeps per unit
        plan = F.Plan(shapes_of(case), case.get("R", 1), case.get("layout", "per_param"))
        mu = F.Muon(plan, [p for p, _, _, _ in places(case)])
        mu.prepare()
        if op == "momentum":
            state["call"] = F.bind_muon_momentum(mu, HP, state["grads"], state["m"],
                                                 state["update"])
        elif op == "orthogonalize":
            state["call"] = F.bind_orthogonalize(mu, HP, state["update"], state["ortho"],
                                                 mu.workspace(state["update"].dtype,
                                                              state["ortho"].dtype))
        else:
            state["call"] = F.bind_muon_apply(mu, HP, state["ortho"], state["master"],
                                              state["param"])
    return state


# --------------------------------------------------------------------- runs
def newton_schulz(X):
    """`steps` products on a batch of matrices of no more rows than columns."""
    a, b, c = HP["coefficients"]
    # |X|_F in 64 bits: sums of up to 59M squares
    X = X * (1.0 / (X.double().square().sum((-2, -1), keepdim=True).sqrt() + HP["eps"])).float()
    for _ in range(HP["steps"]):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return X


def plain(state):
    case, op = state["case"], state["case"]["op"]
    if op == "momentum":
        mu, R = HP["momentum"], case["R"]
        mean = torch.stack([g.float() for g in state["grads"]]).sum(0) / R
        g = [mean[at:at + r * c].view(r, c) for _, at, r, c in places(case)]
        m = [mu * x + (1 - mu) * y for x, y in zip(take_full(case, state["m"]), g)]
        put_full(case, state["m"], m)
        [state["update"][at:at + r * c].copy_(((1 - mu) * y + mu * x).view(-1))
         for (_, at, r, c), x, y in zip(places(case), m, g)]
        return {"m": state["m"], "update": state["update"]}
    if op == "orthogonalize":
        # matrices of one shape go through the products as one batch
        groups = {}
        [groups.setdefault((r, c), []).append(at) for _, at, r, c in places(case)]

        def group(r, c, ats):
            X = torch.stack([state["update"][at:at + r * c].view(r, c) for at in ats]).float()
            X = newton_schulz(X.mT.contiguous()).mT if r > c else newton_schulz(X)
            [state["ortho"][at:at + r * c].view(r, c).copy_(x) for at, x in zip(ats, X)]

        [group(r, c, ats) for (r, c), ats in groups.items()]
        return {"ortho": state["ortho"]}
    lr, wd = HP["lr"], HP["weight_decay"]
    p = [x * (1 - lr * wd) - (lr * 0.2 * math.sqrt(max(r, c))) *
         state["ortho"][at:at + r * c].view(r, c).float()
         for (_, at, r, c), x in zip(places(case), take_full(case, state["master"]))]
    put_full(case, state["master"], p)
    put_full(case, state["param"], p)
    return {"master": state["master"], "param": state["param"]}


def run(state):
    if not own:
        return plain(state)
    state["call"]()
    op = state["case"]["op"]
    if op == "momentum":
        return {"m": state["m"], "update": state["update"]}
    if op == "orthogonalize":
        return {"ortho": state["ortho"]}
    return {"master": state["master"], "param": state["param"]}


# --------------------------------------------------------------------- work
def work(case):
    es = {"bf16": 2, "f32": 4}
    n = sum(r * c for _, _, r, c in places(case))
    if case["op"] == "momentum":
        return {"bytes": n * (case["R"] * es[case["grad"]] + 8 + es[case["update"]]),
                "flops": n * (case["R"] + 6)}
    if case["op"] == "apply":
        return {"bytes": n * (es[case["ortho"]] + 8 + es[case["param"]]), "flops": 3 * n}
    # per step and matrix of m <= k: half of X X^T and of A A (both are
    # symmetric), and the product with X
    flops = sum(HP["steps"] * (3 * min(r, c) ** 2 * max(r, c) + min(r, c) ** 3)
                for _, _, r, c in places(case))
    return {"bytes": n * (es[case["update"]] + es[case["ortho"]]), "flops": flops}


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


def exact(case, seed):
    global own
    kept, own = own, False
    state = prepare(case, seed)
    own = kept
    index = shard_index(case) if "R" in case else None
    if case["op"] == "momentum":
        m, u, mu = state["m"].double(), state["update"].double(), HP["momentum"]
        for _, at, r, c in places(case):
            here = slice(at, at + r * c)
            g = torch.zeros(r * c, dtype=torch.float64, device="cuda")
            for one in state["grads"]:
                g += one[here]
            g /= case["R"]
            new = m[index[here]] * mu + g * (1 - mu)
            m[index[here]] = new
            u[here] = g * (1 - mu) + new * mu
        return {"m": m, "update": u}
    if case["op"] == "orthogonalize":
        a, b, c5 = HP["coefficients"]
        out = torch.zeros(total(case), dtype=torch.float64, device="cuda")
        for _, at, r, c in places(case):
            X = state["update"][at:at + r * c].double().view(r, c)
            X = X / (torch.linalg.norm(X) + HP["eps"])
            for _ in range(HP["steps"]):
                # a X + b (X X^T) X + c (X X^T)^2 X on the shorter side
                if r > c:
                    G = X.T @ X
                    Y = X @ G
                    X = a * X + b * Y + c5 * (Y @ G)
                else:
                    G = X @ X.T
                    Y = G @ X
                    X = a * X + b * Y + c5 * (G @ Y)
            out[at:at + r * c] = X.reshape(-1)
        return {"ortho": out}
    master = state["master"].double()
    param = state["param"].double()
    for _, at, r, c in places(case):
        where = index[at:at + r * c]
        master[where] = (master[where] * (1 - HP["lr"] * HP["weight_decay"]) -
                         HP["lr"] * 0.2 * math.sqrt(max(r, c)) *
                         state["ortho"][at:at + r * c].double())
        param[where] = master[where]
    return {"master": master, "param": param}
