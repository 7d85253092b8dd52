"""Operators around the routed expert layer: what is measured, in plain form and through the library.

The norm in front of a layer (with the residual's addition, and with an output in 8 bits), tokens sorted by
expert and back with their weights, the router's gradient, and the gradients of the others.  Shapes are those
of the Mixtral- and Qwen-shaped layers of this repository (H = 4096, E = 8, top-2 and H = 2048, E = 60, top-4).

`run` with `own` false computes each operator with elementary torch operations in 32 bits; with `own` true it
makes the library's calls.  `exact` computes the definitions in 64 bits.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
EPS = 1e-5
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100
GROUP = 128


def norm(T, H, dtype, out="same", group=0, residual=True, pad=0):
    return {"op": "norm", "T": T, "H": H, "dtype": dtype, "out": out, "group": group, "residual": residual, "pad": pad}


def norm_grad(T, H, dtype, residual=True, pad=0):
    return {"op": "norm_grad", "T": T, "H": H, "dtype": dtype, "residual": residual, "pad": pad}


def moe(op, T, H, E, k, dtype, router="softmax", drop="none", pad=0):
    return {"op": op, "T": T, "H": H, "E": E, "k": k, "dtype": dtype, "router": router, "drop": drop, "pad": pad}


def listed():
    return [
        # a single token's norm in front of a Qwen-shaped layer: latency alone
        dict(norm(1, 2048, "f16"), name="norm decode"),
        # a batch of decoding requests whose next projection takes 8 bits
        dict(norm(256, 4096, "bf16", out="e4m3", group=GROUP), name="norm 8 bits batch"),
        # a prompt in front of a Mixtral-shaped layer
        dict(norm(4096, 4096, "f16"), name="norm prompt"),
        # a training batch's backward pass through the norm and the residual's addition
        dict(norm_grad(16384, 4096, "bf16"), name="norm gradient"),
        # four decoding tokens sent to their experts
        dict(moe("permute", 4, 2048, 60, 4, "f16"), name="permute decode"),
        # a prompt's tokens in 8 bits with their scales, as they are sent to other ranks
        dict(moe("permute", 4096, 4096, 8, 2, "e4m3"), name="permute 8 bits prompt"),
        # a large batch of a skewed router
        dict(moe("permute", 32768, 2048, 60, 4, "bf16", router="zipf"), name="permute batch"),
        # batched decoding with padded requests at the end
        dict(moe("unpermute", 256, 2048, 60, 4, "f16", drop="pad"), name="unpermute batch decode"),
        # ragged prompts joined, back from the experts
        dict(moe("unpermute", 16383, 4096, 8, 2, "bf16"), name="unpermute prompts"),
        # backward pass of the weighted sum: the rows' gradients and the weights'
        dict(moe("unpermute_grad", 8191, 2048, 60, 4, "f16", router="zipf"), name="unpermute gradient"),
        # a small calibration batch through the router's gradient
        dict(moe("router_grad", 256, 2048, 60, 4, "f16"), name="router gradient small"),
        # a training batch through the router's gradient
        dict(moe("router_grad", 16384, 4096, 8, 2, "f16"), name="router gradient batch"),
    ]


def log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "permute", "unpermute", "permute_grad", "unpermute_grad", "router_grad"])
    dtype = rng.choice(["f16", "bf16", "f32"])
    H = 32 * log_uniform(rng, 2, 256)
    T = log_uniform(rng, 1, 32768)
    pad = rng.choice([0, 0, 64])
    if op == "norm" or op == "norm_grad":
        while T * H * BYTES[dtype] > 16384 * 4096 * 2:
            T = T // 2 + 1
        residual = rng.random() < 0.75
        if op == "norm_grad":
            return norm_grad(T, H, dtype, residual, pad)
        out = rng.choice(["same", "e4m3"])
        return norm(T, H, dtype, out, rng.choice([0, GROUP]) if out == "e4m3" else 0, residual, pad)
    E = log_uniform(rng, 4, 256)
    k = rng.randint(1, min(8, E))
    if op == "permute":
        dtype = rng.choice(["f16", "bf16", "f32", "e4m3"])
    if op == "router_grad":
        dtype = "f16"
        while T * H > 16384 * 4096:
            T = T // 2 + 1
    while T * k * H * BYTES[dtype] > 16384 * 4 * 2048 * 2:
        T = T // 2 + 1
    drop = rng.choice(["none", "pad", "none" if op == "router_grad" else "rank"])
    return moe(op, T, H, E, k, dtype, rng.choice(["softmax", "zipf"]), drop, 0 if op == "router_grad" else pad)


def work(case):
    T, H = case["T"], case["H"]
    size = BYTES[case["dtype"]]
    if case["op"] == "norm":
        # x, the residual in and out, the weight; the output and its scales
        moved = T * H * size * (3 if case["residual"] else 1) + H * size
        if case["out"] == "e4m3":
            moved += T * H + 4 * T * (-(-H // case["group"]) if case["group"] else 1)
        else:
            moved += T * H * size
        return {"bytes": moved, "flops": 6 * T * H}
    if case["op"] == "norm_grad":
        return {"bytes": T * H * size * (4 if case["residual"] else 3) + H * (size + 4), "flops": 12 * T * H}
    E, k = case["E"], case["k"]
    S = T * k
    if case["drop"] == "pad":
        live_tokens = T - T // 8
        live = live_tokens * k
    elif case["drop"] == "rank":
        live_tokens, live = T, S // 2
    else:
        live_tokens, live = T, S
    if case["op"] == "permute":
        moved = (live_tokens + live) * H * size + 8 * S + 4 * live + 4 * (E + 1)
        if case["dtype"] == "e4m3":
            moved += (live_tokens + live) * 4 * -(-H // GROUP)
        return {"bytes": moved, "flops": 0}
    if case["op"] == "unpermute":
        return {"bytes": (T + live) * H * size + 8 * S, "flops": 2 * live * H}
    if case["op"] == "permute_grad":
        return {"bytes": (T + live) * H * size + 4 * S, "flops": live * H}
    if case["op"] == "unpermute_grad":
        return {"bytes": (live_tokens + 2 * live) * H * size + 12 * S, "flops": 3 * live * H}
    # router_grad: x, the gradient that is added to and the sum, the router's matrix and its gradient, ids, weights and their gradients
    return {"bytes": 3 * T * H * 2 + E * H * (2 + 4) + 12 * S, "flops": 4 * live * H}


def rows(g, T, H, dtype, pad, std=1.0):
    """T rows of H normal values, `pad` columns apart from each other in a wider matrix."""
    wide = torch.randn((T, H + pad), generator=g, device="cuda", dtype=torch.float32) * std
    return wide.to(DTYPES[dtype])[:, :H]


def empty(T, H, dtype, pad):
    return torch.zeros((T, H + pad), dtype=torch.uint8 if dtype == "e4m3" else DTYPES[dtype], device="cuda").view(DTYPES[dtype])[:, :H]


def routing(g, case):
    """Expert ids (int32 [T][k]) and weights (fp32 [T][k]) of a top-k softmax router; dropped slots hold -1."""
    T, E, k = case["T"], case["E"], case["k"]
    if case["router"] == "zipf":
        p = (torch.randperm(E, generator=g, device="cuda").double() + 1).pow(-1.1)
        u = torch.rand((T, E), generator=g, device="cuda", dtype=torch.float64).clamp(1e-12, 1 - 1e-12)
        logits = ((p / p.sum()).log() - (-u.log()).log()).float()
    else:
        logits = torch.randn((T, E), generator=g, device="cuda")
    top, ids = logits.topk(k, dim=1)
    w = torch.softmax(top, dim=1)
    ids = ids.int()
    if case["drop"] == "pad":      # requests that pad the batch
        ids[T - T // 8:] = -1
    elif case["drop"] == "rank":   # experts that another rank holds
        ids[ids >= (E + 1) // 2] = -1
    return ids.contiguous(), w.contiguous()


def sorted_places(ids, E):
    """Order of the slots by expert (stable; dropped ones last), the first place of each expert, and each slot's place or -1."""
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < E)
    key = torch.where(kept, flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    inv = torch.where(kept, place, torch.full_like(place, -1))
    ends = torch.searchsorted(key[order], torch.arange(E + 1, device=order.device))
    return order, ends.int(), inv.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, T, H, dtype, pad = case["op"], case["T"], case["H"], case["dtype"], case["pad"]
    s = {"op": op, "T": T, "H": H}
    if op in ("norm", "norm_grad"):
        s["weight"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(DTYPES[dtype])
        # a residual stream: a few columns are many times the others
        column = torch.where(torch.rand(H, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        stream = (torch.randn((T, H), generator=g, device="cuda") * column).to(DTYPES[dtype])
        if op == "norm":
            s["x"] = rows(g, T, H, dtype, pad)
            s["residual"] = stream if case["residual"] else None
            s["sum"] = torch.empty_like(stream) if case["residual"] else None
            s["e4m3"] = case["out"] == "e4m3"
            s["y"] = empty(T, H, "e4m3" if s["e4m3"] else dtype, 0)
            s["group"] = case["group"]
            groups = -(-H // case["group"]) if case["group"] else 1
            s["scale"] = torch.zeros((T, groups), dtype=torch.float32, device="cuda") if s["e4m3"] else None
        else:
            s["dy"] = rows(g, T, H, dtype, pad, 0.01)
            s["stream"] = stream
            s["dres"] = rows(g, T, H, dtype, 0, 0.01) if case["residual"] else None
            s["dx"] = torch.empty_like(stream)
            s["dweight"] = torch.empty(H, dtype=torch.float32, device="cuda")
        return s
    E, k = case["E"], case["k"]
    S = T * k
    s |= {"E": E, "k": k}
    s["ids"], s["w"] = routing(g, case)
    if op == "router_grad":
        s["x"] = rows(g, T, H, dtype, 0)
        s["router_w"] = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).half()
        s["dw"] = 0.1 * torch.randn((T, k), generator=g, device="cuda")
        s["dx_add"] = rows(g, T, H, dtype, 0, 0.01)
        s["dx"] = torch.empty_like(s["dx_add"])
        s["drouter_w"] = torch.empty((E, H), dtype=torch.float32, device="cuda")
        return s
    if op == "permute":
        s["x"] = rows(g, T, H, dtype, pad)
        s["xs"] = empty(S, H, dtype, 0)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["inv"] = torch.empty(S, dtype=torch.int32, device="cuda")
        s["perm"] = torch.full((S,), -1, dtype=torch.int32, device="cuda")
        s["x_scale"] = s["xs_scale"] = None
        if dtype == "e4m3":
            groups = -(-H // GROUP)
            s["x_scale"] = 0.01 * (1 + torch.rand((T, groups), generator=g, device="cuda"))
            s["xs_scale"] = torch.zeros((S, groups), dtype=torch.float32, device="cuda")
        return s
    s["inv"] = sorted_places(s["ids"], E)[2]
    if op == "unpermute":
        s["rows"] = rows(g, S, H, dtype, pad)
        s["y"] = empty(T, H, dtype, 0)
    elif op == "permute_grad":
        s["drows"] = rows(g, S, H, dtype, pad, 0.01)
        s["dx"] = empty(T, H, dtype, 0)
    else:
        s["dy"] = rows(g, T, H, dtype, pad, 0.01)
        s["rows"] = rows(g, S, H, dtype, 0)
        s["drows"] = empty(S, H, dtype, 0)
        s["dw"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


# ----- the plain forms ------------------------------------------------------

def run_plain(s):
    return {"norm": plain_norm, "norm_grad": plain_norm_grad, "permute": plain_permute, "unpermute": plain_unpermute,
            "permute_grad": plain_permute_grad, "unpermute_grad": plain_unpermute_grad, "router_grad": plain_router_grad}[s["op"]](s)


def plain_norm(s):
    x = s["x"]
    r = x.float()
    out = {}
    if s["residual"] is not None:
        r = r + s["residual"].float()
        out["sum"] = r.to(x.dtype)
    y = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    if not s["e4m3"]:
        out["y"] = y.to(x.dtype)
        return out
    T, H = y.shape
    group = s["group"] or H
    groups = -(-H // group)
    if groups * group != H:
        y = torch.nn.functional.pad(y, (0, groups * group - H))
    y = y.reshape(T, groups, group)
    scale = (y.abs().amax(dim=2) / E4M3_MAX).clamp(min=SCALE_MIN)
    code = (y / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    out["y"] = code.reshape(T, groups * group)[:, :H]
    out["scale"] = scale
    return out


def plain_norm_grad(s):
    r, dy, H = s["stream"].float(), s["dy"].float(), s["H"]
    rstd = torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS)
    gdy = dy * s["weight"].float()
    dx = rstd * (gdy - r * (rstd * rstd * (gdy * r).sum(dim=1, keepdim=True) / H))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["stream"].dtype), "dweight": (dy * r * rstd).sum(dim=0)}


def plain_permute(s):
    k, S = s["k"], s["T"] * s["k"]
    order, offsets, inv = sorted_places(s["ids"], s["E"])
    at = torch.arange(S, device="cuda") < offsets[-1]
    x = s["x"]
    bits = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
    moved = bits[order // k]
    out = {"offsets": offsets, "inv": inv, "perm": torch.where(at, order, torch.full_like(order, -1)).int(),
           "xs": torch.where(at[:, None], moved, torch.zeros_like(moved)).view(x.dtype)}
    if s["x_scale"] is not None:
        out["xs_scale"] = torch.where(at[:, None], s["x_scale"][order // k], 0.0)
    return out


def gathered(rows_, inv, T, k):
    """The rows of each token's slots in 32 bits, zero for dropped ones: [T][k][H]."""
    kept = inv >= 0
    got = rows_[inv.clamp(min=0).long()].float()
    return torch.where(kept[:, None], got, torch.zeros_like(got)).reshape(T, k, -1)


def plain_unpermute(s):
    return {"y": (gathered(s["rows"], s["inv"], s["T"], s["k"]) * s["w"][:, :, None]).sum(dim=1).to(s["rows"].dtype)}


def plain_permute_grad(s):
    return {"dx": gathered(s["drows"], s["inv"], s["T"], s["k"]).sum(dim=1).to(s["drows"].dtype)}


def plain_unpermute_grad(s):
    T, k, H, S = s["T"], s["k"], s["H"], s["T"] * s["k"]
    dy = s["dy"].float()
    dw = (gathered(s["rows"], s["inv"], T, k) * dy[:, None, :]).sum(dim=2)
    drows = torch.zeros((S + 1, H), dtype=s["rows"].dtype, device="cuda")
    drows[torch.where(s["inv"] >= 0, s["inv"], S).long()] = (s["w"][:, :, None] * dy[:, None, :]).reshape(S, H).to(drows.dtype)
    return {"drows": drows[:S], "dw": dw}


def plain_router_grad(s):
    T, E, w = s["T"], s["E"], s["w"]
    kept = (s["ids"] >= 0) & (s["ids"] < E)
    wdw = torch.where(kept, w * s["dw"], 0.0)
    dlogit = torch.where(kept, wdw - w * wdw.sum(dim=1, keepdim=True), 0.0)
    dense = torch.zeros((T, E + 1), dtype=torch.float32, device="cuda")
    dense.scatter_add_(1, torch.where(kept, s["ids"], E).long(), dlogit)
    dense = dense[:, :E]
    dx = dense @ s["router_w"].float() + s["dx_add"].float()
    return {"dx": dx.half(), "drouter_w": dense.t() @ s["x"].float()}


# ----- the library's calls --------------------------------------------------

def run_own(s):
    from any_precision_bitplane_amd import binding as B
    op, T, H = s["op"], s["T"], s["H"]
    if op == "norm":
        B.pw_rmsnorm(T, H, s["x"], s["weight"], EPS, s["y"], residual=s["residual"], residual_out=s["sum"],
                     scale=s["scale"], group=s["group"])
        out = {"y": s["y"]}
        if s["sum"] is not None:
            out["sum"] = s["sum"]
        if s["scale"] is not None:
            out["scale"] = s["scale"]
        return out
    if op == "norm_grad":
        if "ws" not in s:
            s["ws"] = torch.empty(B.pw_rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
        B.pw_rmsnorm_backward(T, H, s["dy"], s["stream"], s["weight"], EPS, s["dx"], s["dweight"], s["ws"],
                              dresidual=s["dres"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if "shape" not in s:
        s["shape"] = B.shape(H, 32, s["E"], s["k"])
    shape = s["shape"]
    if op == "permute":
        if "ws" not in s:
            s["ws"] = torch.empty(B.pw_moe_permute_workspace_bytes(shape, T), dtype=torch.uint8, device="cuda")
        B.pw_moe_permute(shape, T, s["x"], s["ids"], s["xs"], s["offsets"], s["inv"], s["perm"], s["ws"],
                         x_scale=s["x_scale"], xs_scale=s["xs_scale"])
        out = {n: s[n] for n in ("xs", "offsets", "inv", "perm")}
        if s["xs_scale"] is not None:
            out["xs_scale"] = s["xs_scale"]
        return out
    if op == "unpermute":
        B.pw_moe_unpermute(shape, T, s["rows"], s["inv"], s["w"], s["y"])
        return {"y": s["y"]}
    if op == "permute_grad":
        B.pw_moe_permute_backward(shape, T, s["drows"], s["inv"], s["dx"])
        return {"dx": s["dx"]}
    if op == "unpermute_grad":
        B.pw_moe_unpermute_backward(shape, T, s["dy"], s["rows"], s["inv"], s["w"], s["drows"], s["dw"])
        return {"drows": s["drows"], "dw": s["dw"]}
    if "ws" not in s:
        s["ws"] = torch.empty(B.pw_router_backward_workspace_bytes(shape, T), dtype=torch.uint8, device="cuda")
    B.pw_router_backward(shape, T, s["x"], s["router_w"], s["ids"], s["w"], s["dw"], s["dx"], s["drouter_w"], s["ws"],
                         dx_add=s["dx_add"])
    return {"dx": s["dx"], "drouter_w": s["drouter_w"]}


# ----- the definitions in 64 bits -------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, T, H = s["op"], s["T"], s["H"]
    if op == "norm":
        total = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        rms = (total.pow(2).sum(1) / H + EPS).sqrt()
        y = total / rms.unsqueeze(1) * s["weight"].double()
        out = {} if s["residual"] is None else {"sum": total}
        if s["e4m3"]:
            pieces = y.split(s["group"] or H, dim=1)
            scale = torch.stack([p.abs().max(1).values / 448 for p in pieces], dim=1).clamp(min=2.0 ** -100)
            out["scale"] = scale
            y = y / scale.repeat_interleave(s["group"] or H, dim=1)[:, :H]
        out["y"] = y
        return out
    if op == "norm_grad":
        # dx_i = g_i dy_i / rms - r_i <g dy, r> / (H rms^3), and dweight_i = sum over tokens of dy_i r_i / rms
        r, dy, gain = s["stream"].double(), s["dy"].double(), s["weight"].double()
        rms = (r.pow(2).sum(1, keepdim=True) / H + EPS).sqrt()
        dot = torch.einsum("th,th,h->t", dy, r, gain).unsqueeze(1)
        dx = gain * dy / rms - r * dot / (H * rms.pow(3))
        if s["dres"] is not None:
            dx += s["dres"].double()
        return {"dx": dx, "dweight": torch.einsum("th,th->h", dy, r / rms)}
    E, k = s["E"], s["k"]
    if op == "router_grad":
        # w = softmax over the token's slots: dlogit = (diag(w) - w w^T) dw, and each logit is <x_t, router_w_e>
        kept = (s["ids"] >= 0).double()
        w, dw = s["w"].double() * kept, s["dw"].double() * kept
        dlogit = w * dw - w * torch.einsum("tj,tj->t", w, dw).unsqueeze(1)
        where = s["ids"].clamp(min=0).long()
        dx, drouter = s["dx_add"].double(), torch.zeros((E, H), dtype=torch.float64, device="cuda")
        x, matrix = s["x"].double(), s["router_w"].double()
        for j in range(k):
            dx += dlogit[:, j, None] * matrix[where[:, j]]
            drouter.index_add_(0, where[:, j], dlogit[:, j, None] * x)
        return {"dx": dx, "drouter_w": drouter}
    if op == "permute":
        # the slots of expert 0 in slot order, then those of expert 1, ...; whole numbers have no 64-bit value
        ids = s["ids"].reshape(-1).cpu()
        slots = torch.cat([(ids == e).nonzero().squeeze(1) for e in range(E)]).to("cuda")
        out = {"xs": torch.zeros((T * k, H), dtype=torch.float64, device="cuda")}
        out["xs"][:len(slots)] = s["x"].to(torch.float32)[slots // k].double()
        if s["x_scale"] is not None:
            out["xs_scale"] = torch.zeros(s["xs_scale"].shape, dtype=torch.float64, device="cuda")
            out["xs_scale"][:len(slots)] = s["x_scale"].double()[slots // k]
        return out | {"offsets": None, "inv": None, "perm": None}
    if op in ("unpermute", "permute_grad"):
        source = s["rows"] if op == "unpermute" else s["drows"]
        y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        inv = s["inv"].reshape(T, k)
        for j in range(k):
            at = (inv[:, j] >= 0).nonzero().squeeze(1)
            part = source[inv[at, j].long()].double()
            y[at] += part * s["w"][at, j, None].double() if op == "unpermute" else part
        return {"y" if op == "unpermute" else "dx": y}
    drows = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    inv, dy = s["inv"].reshape(T, k), s["dy"].double()
    for j in range(k):
        at = (inv[:, j] >= 0).nonzero().squeeze(1)
        place = inv[at, j].long()
        drows[place] = s["w"][at, j, None].double() * dy[at]
        dw[at, j] = (s["rows"][place].double() * dy[at]).sum(1)
    return {"drows": drows, "dw": dw}
