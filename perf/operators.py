"""The operators between two edge convolutions, case by case: group norm with an activation on node
rows (forward and backward), 8-bit activation checkpoints, and both in one training step.

Node rows are [n][(lmax + 1)^2][channels], channels last; `structs` structures lie one after another
in the rows, and `pad` rows behind the last one belong to none.
"""
import numpy as np
import torch

own = False

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BLOCK = 32          # values that share a checkpoint scale
EPS = 1e-5


def listed():
    return [
        # one 21-atom molecule, the step of a molecular-dynamics run: latency
        dict(name="norm_molecule", op="norm", nodes=21, structs=1, pad=0, lmax=2, channels=64, groups=8, type="float32", act="silu"),
        # a training batch of small molecules of uneven sizes, a few rows of padding behind
        dict(name="norm_batch", op="norm", nodes=12288, structs=512, pad=37, lmax=2, channels=64, groups=8, type="float32", act="silu"),
        # one periodic cell of 32768 atoms, 128 channels up to rank 2
        dict(name="norm_cell_32k", op="norm", nodes=32768, structs=1, pad=0, lmax=2, channels=128, groups=16, type="float32", act="silu"),
        # scalar channels only, in 16 bits, no activation, an odd number of groups
        dict(name="norm_scalars_bf16", op="norm", nodes=60001, structs=75, pad=0, lmax=0, channels=252, groups=7, type="bfloat16", act="none"),
        # the 1000-atom diamond cell, gradients from the 32-bit input
        dict(name="back_cell_1k", op="back", nodes=1000, structs=1, pad=0, lmax=2, channels=64, groups=8, type="float32", act="silu", keep="none"),
        # the same step for eight cells of 1000 atoms, rank 3, 128 channels, from the int8 checkpoint
        dict(name="back_cells_int8", op="back", nodes=8000, structs=8, pad=0, lmax=3, channels=128, groups=16, type="float32", act="silu", keep="int8"),
        # odd channels, 16 bits, structures of a few atoms with empty ones among them, from the e4m3 checkpoint
        dict(name="back_odd_e4m3", op="back", nodes=20011, structs=4000, pad=5, lmax=1, channels=50, groups=5, type="float16", act="silu", keep="e4m3"),
        # the features of the 1000-atom cell, kept and fetched again
        dict(name="keep_cell_1k", op="keep", nodes=1000, cols=576, type="float32", keep="int8"),
        # the features of an 8000-atom cell at rank 3 with 128 channels
        dict(name="keep_cell_8k", op="keep", nodes=8000, cols=2048, type="float32", keep="int8"),
        # rows that end inside a block of 32, 16 bits
        dict(name="keep_odd_bf16", op="keep", nodes=16411, cols=1153, type="bfloat16", keep="e4m3"),
        # forward and backward of one training step, 8000 atoms at rank 3, the input kept in int8
        dict(name="step_cells_int8", op="step", nodes=8000, structs=8, pad=0, lmax=3, channels=128, groups=16, type="float32", act="silu", keep="int8"),
        # the same for a batch of molecules, e4m3, 16 bits
        dict(name="step_batch_e4m3", op="step", nodes=12289, structs=600, pad=0, lmax=2, channels=96, groups=12, type="bfloat16", act="silu", keep="e4m3"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    kind = rng.choice(["float32", "float32", "bfloat16", "float16"])
    op = rng.choice(["norm", "norm", "back", "back", "keep", "step"])
    if op == "keep":
        cols = log(1, 2048)
        return dict(op=op, nodes=log(1, max(1, min(60000, 16000000 // cols))), cols=cols, type=kind, keep=rng.choice(["int8", "e4m3"]))
    lmax = rng.randint(0, 3)
    channels = rng.choice([32, 64, 96, 128, 4 * rng.randint(1, 64), rng.randint(4, 256)])
    groups = rng.choice([g for g in range(1, channels + 1) if channels % g == 0 and channels // g >= 4 and g <= 64])
    nodes = log(1, max(1, min(40000, 16000000 // (channels * (lmax + 1) ** 2))))
    structs = log(1, max(1, min(4000, nodes)))
    case = dict(op=op, nodes=nodes, structs=structs, pad=rng.choice([0, 0, min(nodes - 1, rng.randint(1, 40))]), lmax=lmax, channels=channels, groups=groups, type=kind, act=rng.choice(["silu", "silu", "none"]))
    if op != "norm":
        case["keep"] = rng.choice(["int8", "e4m3"] if op == "step" else ["none", "int8", "e4m3"])
    return case


def _ranks(lmax, device):
    """Rank of each of the (lmax + 1)^2 components."""
    return torch.arange((lmax + 1) ** 2, device=device).double().add(0.5).sqrt().long()


def _features(case, rows, cols, gen):
    """Features as a layer leaves them: each column a scale and an offset of its own, a few rows far out."""
    dev = gen.device
    x = torch.randn(rows, cols, generator=gen, device=dev)
    scale = torch.randn(cols, generator=gen, device=dev).mul(0.5).exp()
    shift = torch.randn(cols, generator=gen, device=dev).mul(0.3)
    far = torch.rand(rows, 1, generator=gen, device=dev).pow(6).mul(2).add(0.7)
    return (x * scale * far + shift).to(TYPES[case["type"]])


def _node_ptr(case, seed):
    """Starts of the structures: cells of one size where the rows are few per structure's end, else uneven, some empty."""
    n, s = case["nodes"] - case["pad"], case["structs"]
    rng = np.random.default_rng([seed, 9])
    cuts = np.sort(rng.integers(0, n + 1, s - 1))
    if n >= 500 * s:
        cuts = np.arange(1, s) * n // s
    return torch.from_numpy(np.concatenate([[0], cuts, [n]]).astype(np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case=case)
    if case["op"] == "keep":
        state["x"] = _features(case, case["nodes"], case["cols"], gen)
        return state
    k, c = (case["lmax"] + 1) ** 2, case["channels"]
    state["x"] = _features(case, case["nodes"], k * c, gen)
    state["node_ptr"] = _node_ptr(case, seed)
    state["weight"] = 1 + 0.2 * torch.randn(case["lmax"] + 1, c, generator=gen, device="cuda")
    state["bias"] = 0.2 * torch.randn(c, generator=gen, device="cuda")
    if case["op"] != "norm":
        state["grad"] = torch.randn(case["nodes"], k * c, generator=gen, device="cuda").to(TYPES[case["type"]])
    if case["op"] == "back":   # what the forward left: the statistics, and the checkpoint in the input's place
        state["stats"] = _forward(state)[1]
        if case["keep"] != "none":
            state["codes"], state["scale"] = _store(state["x"], case["keep"])
            del state["x"]
    return state


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "norm":
        return _forward(state)
    if case["op"] == "keep":
        codes, scale = _store(state["x"], case["keep"])
        return _restore(codes, scale, state["x"].dtype)
    if case["op"] == "back":
        x = state["x"] if case["keep"] == "none" else _restore(state["codes"], state["scale"], torch.float32)
        return _backward(state, x, state["stats"])
    codes, scale = _store(state["x"], case["keep"])
    y, stats = _forward(state)
    return (y, stats) + _backward(state, _restore(codes, scale, torch.float32), stats)


def _run_own(case, state):
    import equivariant_mlip_tensor_edge_b200 as etp

    if case["op"] == "keep":
        return etp.checkpoint8(state["x"], case["keep"]).restore()
    args = dict(lmax=case["lmax"], groups=case["groups"], node_ptr=state["node_ptr"], activation=case["act"])
    if case["op"] == "norm":
        return etp.group_norm(state["x"], state["weight"], state["bias"], eps=EPS, **args)[:2]
    if case["op"] == "back":
        x = state["x"] if case["keep"] == "none" else etp.Checkpoint8(state["codes"], state["scale"], TYPES[case["type"]])
        return etp.group_norm_backward(x, state["stats"], state["weight"], state["bias"], state["grad"], **args)
    y, stats, kept = etp.group_norm(state["x"], state["weight"], state["bias"], eps=EPS, checkpoint=case["keep"], **args)
    return (y, stats) + etp.group_norm_backward(kept, stats, state["weight"], state["bias"], state["grad"], **args)


# ---- plain forms, 32 bits (64 in the long sums)

def _segments(state):
    """Structure of each row (the number of structures for rows that belong to none), and the rows of each."""
    ptr = state["node_ptr"].long()
    rows = torch.arange(state["case"]["nodes"], device=ptr.device)
    return torch.searchsorted(ptr[1:].contiguous(), rows, right=True), torch.cat([ptr.diff(), ptr.new_ones(1)])


def _group_sums(v, seg, ranks, count):
    """[n, k, g, cg] summed over the channels of a group, the components of a rank and the rows of a structure."""
    per = v.sum(-1, dtype=torch.float64)
    per = per.new_zeros(len(count), *per.shape[1:]).index_add_(0, seg, per)
    return per.new_zeros(len(count), int(ranks.max()) + 1, per.shape[2]).index_add_(1, ranks, per)


def _forward(state):
    case, x = state["case"], state["x"].float()
    n, k, c, g = case["nodes"], (case["lmax"] + 1) ** 2, case["channels"], case["groups"]
    ranks = _ranks(case["lmax"], x.device)
    seg, count = _segments(state)
    x = x.view(n, k, g, c // g)
    size = (count[:, None] * (2 * torch.arange(case["lmax"] + 1, device=x.device) + 1) * (c // g)).clamp(min=1)[..., None]
    mean = (_group_sums(x[:, :1], seg, ranks[:1], count) / size[:, :1]).float()
    x = torch.cat([x[:, :1] - mean[seg][..., None], x[:, 1:]], 1)
    rstd = (_group_sums(x * x, seg, ranks, count) / size + EPS).rsqrt().float()
    rstd = torch.where(count[:, None, None] > 0, rstd, 0.0)
    y = (x * rstd[seg][:, ranks][..., None]).view(n, k, c) * state["weight"][ranks]
    y = torch.cat([y[:, :1] + state["bias"], y[:, 1:]], 1)
    if case["act"] == "silu":
        y = y / (1 + torch.exp(-y[:, :1]))
    y = torch.where((seg < case["structs"])[:, None, None], y, 0.0)
    return y.view(n, k * c).to(state["x"].dtype), torch.cat([mean, rstd], 1)[:-1]


def _backward(state, x, stats):
    case, grad = state["case"], state["grad"].float()
    n, k, c, g = case["nodes"], (case["lmax"] + 1) ** 2, case["channels"], case["groups"]
    ranks = _ranks(case["lmax"], x.device)
    seg, count = _segments(state)
    inside = (seg < case["structs"])[:, None, None]
    grad = torch.where(inside, grad.view(n, k, c), 0.0)
    x = torch.where(inside, x.float().view(n, k, c), 0.0).view(n, k, g, c // g)
    stats = torch.cat([stats, torch.zeros_like(stats[:1])])
    mean, rstd = stats[:, :1], stats[:, 1:][seg][:, ranks][..., None]
    hat = torch.cat([x[:, :1] - mean[seg][..., None], x[:, 1:]], 1) * rstd
    weight = state["weight"][ranks]
    dy = grad
    if case["act"] == "silu":
        y = hat.view(n, k, c) * weight
        y = torch.cat([y[:, :1] + state["bias"], y[:, 1:]], 1)
        gate = 1 / (1 + torch.exp(-y[:, :1]))
        dy = grad * gate
        dy = torch.cat([dy[:, :1] + gate * (1 - gate) * (grad * y).sum(1, keepdim=True), dy[:, 1:]], 1)
    dy = torch.where(inside, dy, 0.0)
    part = (dy * hat.view(n, k, c)).sum(0, dtype=torch.float64)
    grad_weight = part.new_zeros(case["lmax"] + 1, c).index_add_(0, ranks, part).float()
    grad_bias = dy[:, 0].sum(0, dtype=torch.float64).float()
    h = (dy * weight).view(n, k, g, c // g)
    size = (count[:, None] * (2 * torch.arange(case["lmax"] + 1, device=x.device) + 1) * (c // g)).clamp(min=1)[..., None]
    along = (_group_sums(h * hat, seg, ranks, count) / size).float()[seg][:, ranks][..., None]
    level = (_group_sums(h[:, :1], seg, ranks[:1], count) / size[:, :1]).float()[seg][..., None]
    dx = h - hat * along
    dx = torch.cat([dx[:, :1] - level, dx[:, 1:]], 1) * rstd
    return dx.view(n, k * c).to(state["grad"].dtype), grad_weight, grad_bias


def _power(e):
    """2^e in 32 bits, e between -126 and 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _store(x, keep):
    """Codes [n, cols] and scale bytes [n, blocks]: 2^(byte - 127), 255 for a block that is not finite."""
    n, cols = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK)).view(n, -1, BLOCK)
    top = v.abs().amax(-1)
    m, e = torch.frexp(top)
    e = e - 7 + (m > 127 / 128).int() if keep == "int8" else e - 9 + (m > 0.875).int()
    e = torch.where(top > 0, e, -126).clamp(min=-126)
    fine = torch.isfinite(top)
    e = torch.where(fine, e, 0)
    v = torch.where(fine[..., None], v, 0.0) * _power(-e)[..., None]
    codes = v.round().to(torch.int8) if keep == "int8" else v.to(torch.float8_e4m3fn)
    return codes.view(n, -1)[:, :cols].contiguous(), torch.where(fine, e + 127, 255).to(torch.uint8)


def _restore(codes, scale, dtype):
    """Values of the codes, held to the type's finite range; NaN for a block that was not finite."""
    cols = codes.shape[1]
    byte = scale.int().repeat_interleave(BLOCK, 1)[:, :cols]
    most = torch.finfo(dtype).max
    value = (codes.float() * _power(torch.where(byte < 255, byte - 127, 0))).clamp(-most, most)
    return torch.where(byte < 255, value, torch.nan).to(dtype)


# ---- the definition in 64 bits, structure by structure

def _exact_round(v, keep):
    if keep == "int8":
        return torch.round(v)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_kept(x, keep):
    """The values that a checkpoint of x stands for."""
    x = x.double()
    out = torch.zeros_like(x)
    most = 127.0 if keep == "int8" else 448.0
    for j in range(0, x.shape[1], BLOCK):
        v = x[:, j:j + BLOCK]
        top = v.abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(top / most)).clamp(min=-126)
        e = torch.where(top > most * torch.exp2(e), e + 1, e)
        e = torch.where((top <= most * torch.exp2(e - 1)) & (e > -126), e - 1, e)
        out[:, j:j + BLOCK] = _exact_round(v / torch.exp2(e), keep) * torch.exp2(e)
    return out


def _exact_norm(x, state, grad=None, stats=None):
    """Forward (grad None) or backward of one group norm."""
    case = state["case"]
    lmax, c, g = case["lmax"], case["channels"], case["groups"]
    w, b = state["weight"].double().view(lmax + 1, g, c // g), state["bias"].double().view(g, c // g)
    ptr = state["node_ptr"].tolist()
    x = x.double().view(case["nodes"], -1, g, c // g)
    out = torch.zeros_like(x)
    found = x.new_zeros(case["structs"], lmax + 2, g)
    gw, gb = torch.zeros_like(w), torch.zeros_like(b)
    cut = [slice(r * r, (r + 1) ** 2) for r in range(lmax + 1)]
    for s in range(case["structs"]):
        lo, hi = ptr[s], ptr[s + 1]
        if lo == hi:
            continue
        v = x[lo:hi]
        if stats is None:
            found[s, 0] = v[:, 0].mean((0, 2))
            found[s, 1] = (v[:, 0].var((0, 2), correction=0) + EPS) ** -0.5
            for r in range(1, lmax + 1):
                found[s, 1 + r] = (v[:, cut[r]].square().mean((0, 1, 3)) + EPS) ** -0.5
        else:
            found[s] = stats[s].double()
        hat = torch.empty_like(v)
        y = torch.empty_like(v)
        for r in range(lmax + 1):
            hat[:, cut[r]] = (v[:, cut[r]] - (found[s, 0][:, None] if r == 0 else 0)) * found[s, 1 + r][:, None]
            y[:, cut[r]] = hat[:, cut[r]] * w[r] + (b if r == 0 else 0)
        gate = torch.sigmoid(y[:, :1]) if case["act"] == "silu" else torch.ones_like(y[:, :1])
        if grad is None:
            out[lo:hi] = y * gate
            continue
        go = grad[lo:hi].double().view_as(v)
        dy = go * gate
        if case["act"] == "silu":
            dy[:, 0] += (go * y).sum(1) * (gate * (1 - gate))[:, 0]
        gb += dy[:, 0].sum(0)
        for r in range(lmax + 1):
            h, u = dy[:, cut[r]], hat[:, cut[r]]
            gw[r] += (h * u).sum((0, 1))
            h = h * w[r]
            d = h - u * (h * u).mean((0, 1, 3))[:, None]
            if r == 0:
                d = d - h.mean((0, 1, 3))[:, None]
            out[lo:hi, cut[r]] = d * found[s, 1 + r][:, None]
    out = out.view(case["nodes"], -1)
    return (out, found) if grad is None else (out, gw.view(lmax + 1, c), gb.view(c))


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "keep":
        return _exact_kept(state["x"], case["keep"])
    if case["op"] == "norm":
        return _exact_norm(state["x"], state)
    if case["op"] == "back":
        if case["keep"] == "none":
            x = state["x"]
        else:
            power = torch.exp2(state["scale"].double() - 127)
            x = state["codes"].double() * power.repeat_interleave(BLOCK, 1)[:, :state["codes"].shape[1]]
        return _exact_norm(x, state, state["grad"], state["stats"])
    y, stats = _exact_norm(state["x"], state)
    return (y, stats) + _exact_norm(_exact_kept(state["x"], case["keep"]), state, state["grad"], stats)


def work(case):
    size = 4 if case["type"] == "float32" else 2
    if case["op"] == "keep":   # the input, the checkpoint written and read, the output
        values = case["nodes"] * case["cols"]
        return dict(bytes=values * (2 * size + 2 + 2 / BLOCK), flops=6 * values)
    values = case["nodes"] * case["channels"] * (case["lmax"] + 1) ** 2
    kept = 1 + 1 / BLOCK if case.get("keep", "none") != "none" else size
    small = 4 * (case["structs"] * ((case["lmax"] + 2) * case["groups"] + 1) + (case["lmax"] + 2) * case["channels"])
    forward, backward = dict(bytes=2 * size * values + small, flops=8 * values), dict(bytes=(2 * size + kept) * values + 2 * small, flops=20 * values)
    if case["op"] == "norm":
        return forward
    if case["op"] == "back":
        return backward
    return dict(bytes=forward["bytes"] + kept * values + backward["bytes"], flops=28 * values)
