"""Expert products in 16 bits: what is measured, in plain form and through the library.

Between the tokens sorted by expert and their way back: the gated feed-forward block of every expert (one shared
expert too), a product with bias, activation and residual, their gradients, and gate and up kept for the backward
pass in 16 or in 8 bits.  Shapes are those of the Mixtral- and Qwen-shaped layers of this repository (H = 4096,
I = 14336, E = 8, top-2 and H = 2048, I = 1408, E = 60, top-4).

`run` with `own` false computes each operator with elementary torch operations in 32 bits; with `own` true it
makes the library's calls.  `exact` computes the definitions in 64 bits.
"""
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100
GROUP = 128
SQRT_HALF = 0.5 ** 0.5
INV_SQRT_2PI = 0.3989422804014327
ACTS = {"none": 0, "silu": 1, "gelu": 2}


def ffn(T, H, I, E, k, dtype, router="even", drop="none", act="silu", keep="none", pad=0):
    """keep: how gate and up are kept for the backward pass (not at all, in the rows' type, in 8 bits)."""
    return {"op": "ffn", "T": T, "H": H, "I": I, "E": E, "k": k, "dtype": dtype, "router": router, "drop": drop,
            "act": act, "keep": keep, "pad": pad}


def ffn_grad(T, H, I, E, k, dtype, router="even", drop="none", act="silu", keep="same", pad=0):
    return dict(ffn(T, H, I, E, k, dtype, router, drop, act, keep, pad), op="ffn_grad")


def product(T, N, K, E, k, dtype, router="even", drop="none", act="none", bias=True, residual=False, pre=False, pad=0):
    return {"op": "product", "T": T, "N": N, "K": K, "E": E, "k": k, "dtype": dtype, "router": router, "drop": drop,
            "act": act, "bias": bias, "residual": residual, "pre": pre, "pad": pad}


def product_grad(T, N, K, E, k, dtype, router="even", drop="none", act="none", bias=True, pad=0):
    return dict(product(T, N, K, E, k, dtype, router, drop, act, bias, False, False, pad), op="product_grad")


def listed():
    return [
        # one token through a shared expert four times as wide as a routed one: latency and the weights' bytes
        dict(ffn(1, 2048, 5632, 1, 1, "f16"), name="ffn shared decode"),
        # four decoding requests through their routed experts, one or two rows each
        dict(ffn(4, 2048, 1408, 60, 4, "f16"), name="ffn routed decode"),
        # batched decoding with every expert hit by some rows
        dict(ffn(64, 4096, 14336, 8, 2, "f16"), name="ffn batch decode"),
        # a prompt of a skewed router, its padding dropped
        dict(ffn(4096, 2048, 1408, 60, 4, "bf16", router="skewed", drop="pad"), name="ffn prompt"),
        # a training batch's forward pass, gate and up kept in 8 bits
        dict(ffn(4095, 4096, 14336, 8, 2, "bf16", keep="e4m3"), name="ffn training"),
        # a small calibration batch's gradients
        dict(ffn_grad(256, 2048, 1408, 60, 4, "f16"), name="ffn gradient small"),
        # a training batch of many narrow experts, skewed, from 8-bit checkpoints
        dict(ffn_grad(4096, 2048, 1408, 60, 4, "bf16", router="skewed", keep="e4m3"), name="ffn gradient 8 bits"),
        # a training batch of a few wide experts
        dict(ffn_grad(4096, 4096, 14336, 8, 2, "f16"), name="ffn gradient large"),
        # a projection of a few decoding requests
        dict(product(7, 6144, 4096, 1, 1, "f16"), name="product decode"),
        # experts without a gate on a training batch: bias and activation, the sum kept for the backward pass
        dict(product(4097, 8192, 2048, 8, 2, "bf16", act="gelu", residual=True, pre=True), name="product training"),
        # a projection's gradients on a small ragged batch of prompts
        dict(product_grad(511, 2048, 2048, 1, 1, "f16"), name="product gradient small"),
        # the gradients of the experts without a gate
        dict(product_grad(4097, 8192, 2048, 8, 2, "bf16", act="gelu"), name="product gradient"),
    ]


def log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_grad", "product", "product_grad"])
    dtype = rng.choice(["f16", "bf16"])
    E = rng.choice([1, log_uniform(rng, 2, 64), log_uniform(rng, 2, 64)])
    k = rng.randint(1, min(4, E))
    T = log_uniform(rng, 1, 16384)
    router, drop = rng.choice(["even", "skewed"]), rng.choice(["none", "none", "pad"])
    pad = rng.choice([0, 0, 64])
    if op in ("ffn", "ffn_grad"):
        H, I = 32 * log_uniform(rng, 2, 128), 32 * log_uniform(rng, 2, 448)
        while E * H * I > 8 * 4096 * 14336:
            E = E // 2
        k = min(k, E)
        while T * k * H * I > 8192 * 4096 * 14336:
            T = T // 2 + 1
        act = rng.choice(["silu", "silu", "gelu"])
        if op == "ffn":
            return ffn(T, H, I, E, k, dtype, router, drop, act, rng.choice(["none", "none", "same", "e4m3"]), pad)
        return ffn_grad(T, H, I, E, k, dtype, router, drop, act, rng.choice(["same", "e4m3"]), pad)
    N, K = 8 * log_uniform(rng, 4, 1536), 8 * log_uniform(rng, 4, 1536)
    while E * N * K > 8 * 4096 * 14336:
        E = E // 2
    k = min(k, E)
    while T * k * N * K > 16384 * 4096 * 14336:
        T = T // 2 + 1
    act, bias = rng.choice(["none", "silu", "gelu"]), rng.random() < 0.5
    if op == "product":
        return product(T, N, K, E, k, dtype, router, drop, act, bias, rng.random() < 0.5, rng.random() < 0.25, pad)
    return product_grad(T, N, K, E, k, dtype, router, drop, act, bias, pad)


def kept_tokens(case):
    return case["T"] - case["T"] // 8 if case["drop"] == "pad" else case["T"]


def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    live = kept_tokens(case) * k
    # experts that evenly routed tokens reach (all of them but for a few tokens)
    reached = E * (1 - (1 - k / E) ** kept_tokens(case))
    if case["op"] in ("ffn", "ffn_grad"):
        H, I = case["H"], case["I"]
        groups = 2 * -(-I // GROUP)
        z = {"none": 0, "same": 4 * I, "e4m3": 2 * I + 4 * groups}[case["keep"]]
        if case["op"] == "ffn":
            return {"bytes": int(reached * 3 * H * I * 2 + live * (4 * H + z) + 4 * (E + 1)), "flops": 6 * live * H * I}
        # dy, x, gate and up, the weights; dx and the weights' gradients
        return {"bytes": int(reached * 3 * H * I * 2 + E * 3 * H * I * 2 + live * (6 * H + z) + 4 * (E + 1)),
                "flops": 12 * live * H * I}
    N, K = case["N"], case["K"]
    if case["op"] == "product":
        rows_ = live * 2 * (K + N * (1 + case["residual"] + case["pre"]))
        return {"bytes": int(reached * N * K * 2 + rows_ + 2 * E * N * case["bias"] + 4 * (E + 1)), "flops": 2 * live * N * K}
    rows_ = live * 2 * (2 * K + N * (1 + (case["act"] != "none")))
    return {"bytes": int((reached + E) * N * K * 2 + rows_ + 2 * E * N * case["bias"] + 4 * (E + 1)), "flops": 4 * live * N * K}


def normal(g, shape, dtype, std=1.0):
    out = torch.empty(shape, dtype=DTYPES[dtype], device="cuda")
    return out.normal_(0.0, std, generator=g)


def rows(g, S, H, dtype, pad, std=1.0):
    """S rows of H normal values, `pad` columns apart from each other in a wider matrix."""
    return normal(g, (S, H + pad), dtype, std)[:, :H]


def routing(g, case):
    """Rows of each expert as a sort of the tokens by expert leaves them: offsets int32 [E+1], and the longest expert's length."""
    T, E, k = kept_tokens(case), case["E"], case["k"]
    logits = torch.randn((T, E), generator=g, device="cuda")
    if case["router"] == "skewed":   # some experts are asked for several times as often as others
        logits = logits + torch.randn((1, E), generator=g, device="cuda") * 0.5
    counts = torch.bincount(logits.topk(k, dim=1).indices.reshape(-1), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, int(counts.max())


def pack8(z, I):
    """e4m3 codes and fp32 scales of gate and up ([S][2I]), a scale per 128 columns of each half."""
    S, groups = z.shape[0], -(-I // GROUP)
    z = torch.nn.functional.pad(z.reshape(S, 2, I), (0, groups * GROUP - I)).reshape(S, 2, groups, GROUP)
    scale = (z.abs().amax(dim=3) / E4M3_MAX).clamp(min=SCALE_MIN)
    code = (z / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    code = code.reshape(S, 2, groups * GROUP).view(torch.uint8)[:, :, :I].reshape(S, 2 * I).view(torch.float8_e4m3fn)
    return code, scale.reshape(S, 2 * groups)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dtype, E, pad = case["dtype"], case["E"], case["pad"]
    S = case["T"] * case["k"]
    offsets, longest = routing(g, case)
    dense = E == 1 and case["drop"] == "none"
    s = {"op": case["op"], "S": S, "E": E, "act": case["act"], "dtype": DTYPES[dtype], "longest": longest,
         "offsets": None if dense else offsets}
    if case["op"] in ("ffn", "ffn_grad"):
        H, I = case["H"], case["I"]
        s |= {"H": H, "I": I, "keep": case["keep"]}
        s["x"] = rows(g, S, H, dtype, pad)
        s["w_gate_up"] = normal(g, (E, 2 * I, H), dtype, H ** -0.5)
        s["w_down"] = normal(g, (E, H, I), dtype, I ** -0.5)
        if case["op"] == "ffn":
            s["y"] = torch.zeros((S, H), dtype=DTYPES[dtype], device="cuda")
            s["z"] = s["z_scale"] = None
            if case["keep"] == "same":
                s["z"] = torch.zeros((S, 2 * I), dtype=DTYPES[dtype], device="cuda")
            elif case["keep"] == "e4m3":
                s["z"] = torch.zeros((S, 2 * I), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                s["z_scale"] = torch.zeros((S, 2 * -(-I // GROUP)), dtype=torch.float32, device="cuda")
            return s
        s["dy"] = rows(g, S, H, dtype, pad, 0.01)
        z = normal(g, (S, 2 * I), dtype)
        s["z"], s["z_scale"] = pack8(z.float(), I) if case["keep"] == "e4m3" else (z, None)
        s["dx"] = torch.zeros((S, H), dtype=DTYPES[dtype], device="cuda")
        s["dw_gate_up"], s["dw_down"] = torch.empty_like(s["w_gate_up"]), torch.empty_like(s["w_down"])
        return s
    N, K = case["N"], case["K"]
    s |= {"N": N, "K": K}
    s["x"] = rows(g, S, K, dtype, pad)
    s["w"] = normal(g, (E, N, K), dtype, K ** -0.5)
    s["bias"] = normal(g, (E, N), dtype, 0.2) if case["bias"] else None
    if case["op"] == "product":
        s["residual"] = rows(g, S, N, dtype, pad) if case["residual"] else None
        s["y"] = torch.zeros((S, N), dtype=DTYPES[dtype], device="cuda")
        s["pre"] = torch.zeros_like(s["y"]) if case["pre"] else None
        return s
    s["dy"] = rows(g, S, N, dtype, pad, 0.01)
    s["pre"] = rows(g, S, N, dtype, 0) if case["act"] != "none" else None
    s["dx"] = torch.zeros((S, K), dtype=DTYPES[dtype], device="cuda")
    s["dw"] = torch.empty_like(s["w"])
    s["dbias"] = torch.empty((E, N), dtype=DTYPES[dtype], device="cuda") if case["bias"] else None
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


# ----- the plain forms ------------------------------------------------------

def run_plain(s):
    return {"ffn": plain_ffn, "ffn_grad": plain_ffn_grad, "product": plain_product, "product_grad": plain_product_grad}[s["op"]](s)


class Groups:
    """The rows of every expert side by side, padded to the longest expert's (few rows: every row with its own expert's matrix)."""

    def __init__(self, s):
        S, self.E, self.offsets, self.longest = s["S"], s["E"], s["offsets"], s["longest"]
        self.S = S
        if self.offsets is None:
            return
        at = torch.arange(S, device="cuda")
        self.expert = torch.searchsorted(self.offsets[1:].long(), at, right=True)
        self.kept = self.expert < self.E
        self.expert = self.expert.clamp(max=self.E - 1)
        self.by_row = S <= self.E
        # dropped rows go to a place of their own behind all others
        place = self.expert * self.longest + at - self.offsets.long()[self.expert]
        self.place = torch.where(self.kept, place, self.E * self.longest)

    def spread(self, x):
        """[S][n] to [E][longest][n] in 32 bits, zeros where an expert has fewer rows."""
        if self.offsets is None:
            return x.float()[None]
        out = torch.zeros((self.E * self.longest + 1, x.shape[1]), dtype=torch.float32, device="cuda")
        out[self.place] = x.float()
        return out[:-1].reshape(self.E, self.longest, -1)

    def gather(self, x):
        """Back from spread(): [S][n], zeros in dropped rows."""
        if self.offsets is None:
            return x[0]
        flat = torch.cat([x.reshape(self.E * self.longest, -1), x.new_zeros((1, x.shape[2]))])
        return flat[self.place]

    def times(self, x, w):
        """x [S][K] by each row's expert's w [E][N][K]: [S][N]."""
        if self.offsets is not None and self.by_row:
            y = torch.bmm(w[self.expert].float(), x.float()[:, :, None])[:, :, 0]
            return torch.where(self.kept[:, None], y, 0.0)
        return self.gather(torch.bmm(self.spread(x), w.float().transpose(1, 2)))

    def times_t(self, x, w):
        """x [S][N] by each row's expert's w [E][N][K]: [S][K]."""
        if self.offsets is not None and self.by_row:
            y = torch.bmm(x.float()[:, None, :], w[self.expert].float())[:, 0, :]
            return torch.where(self.kept[:, None], y, 0.0)
        return self.gather(torch.bmm(self.spread(x), w.float()))

    def outer(self, a, b):
        """Sum over each expert's rows of a's outer b: [E][n][m]."""
        return torch.bmm(self.spread(a).transpose(1, 2), self.spread(b))

    def total(self, a):
        """Sum over each expert's rows: [E][n]."""
        return self.spread(a).sum(dim=1)


def plain_act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    return 0.5 * z * (1 + torch.erf(z * SQRT_HALF)) if act == "gelu" else z


def plain_act_grad(z, act):
    if act == "silu":
        sig = torch.sigmoid(z)
        return sig * (1 + z * (1 - sig))
    return 0.5 * (1 + torch.erf(z * SQRT_HALF)) + z * torch.exp(-0.5 * z * z) * INV_SQRT_2PI


def plain_ffn(s):
    I, groups = s["I"], Groups(s)
    z = groups.times(s["x"], s["w_gate_up"])
    out = {"y": groups.times(plain_act(z[:, :I], s["act"]) * z[:, I:], s["w_down"]).to(s["dtype"])}
    if s["keep"] == "same":
        out["z"] = z.to(s["dtype"])
    elif s["keep"] == "e4m3":
        code, scale = pack8(z, I)
        if s["offsets"] is not None:
            code = torch.where(groups.kept[:, None], code.view(torch.uint8), 0).view(torch.float8_e4m3fn)
            scale = torch.where(groups.kept[:, None], scale, 0.0)
        out |= {"z": code, "z_scale": scale}
    return out


def plain_ffn_grad(s):
    I, groups = s["I"], Groups(s)
    z = s["z"].float()
    if s["z_scale"] is not None:
        z = z * torch.repeat_interleave(s["z_scale"].reshape(-1, 2, s["z_scale"].shape[1] // 2), GROUP, dim=2)[:, :, :I].reshape(z.shape)
    gate, up = z[:, :I], z[:, I:]
    dh = groups.times_t(s["dy"], s["w_down"])
    dz = torch.cat([dh * up * plain_act_grad(gate, s["act"]), dh * plain_act(gate, s["act"])], dim=1)
    return {"dx": groups.times_t(dz, s["w_gate_up"]).to(s["dtype"]),
            "dw_gate_up": groups.outer(dz, s["x"]).to(s["dtype"]),
            "dw_down": groups.outer(s["dy"], plain_act(gate, s["act"]) * up).to(s["dtype"])}


def plain_product(s):
    groups = Groups(s)
    z = groups.times(s["x"], s["w"])
    if s["bias"] is not None:
        z = z + (s["bias"].float() if s["offsets"] is None else s["bias"].float()[groups.expert])
    y = plain_act(z, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y} if s["pre"] is None else {"y": y, "pre": z}
    if s["offsets"] is not None:
        out = {n: torch.where(groups.kept[:, None], v, 0.0) for n, v in out.items()}
    return {n: v.to(s["dtype"]) for n, v in out.items()}


def plain_product_grad(s):
    groups = Groups(s)
    dz = s["dy"].float()
    if s["pre"] is not None:
        dz = dz * plain_act_grad(s["pre"].float(), s["act"])
    out = {"dx": groups.times_t(dz, s["w"]).to(s["dtype"]), "dw": groups.outer(dz, s["x"]).to(s["dtype"])}
    if s["dbias"] is not None:
        out["dbias"] = groups.total(dz).to(s["dtype"])
    return out


# ----- the library's calls --------------------------------------------------

def run_own(s):
    from any_precision_bitplane_amd import binding as B
    op, S, E, act = s["op"], s["S"], s["E"], ACTS[s["act"]]
    if op in ("ffn", "ffn_grad"):
        if "shape" not in s:
            s["shape"] = B.shape(s["H"], s["I"], E, 1)
            size = B.pw_moe_ffn_workspace_bytes if op == "ffn" else B.pw_moe_ffn_backward_workspace_bytes
            s["ws"] = torch.empty(size(s["shape"], S), dtype=torch.uint8, device="cuda")
        if op == "ffn":
            B.pw_moe_ffn(s["shape"], S, s["x"], s["w_gate_up"], s["w_down"], s["y"], s["ws"], offsets=s["offsets"],
                         act=act, z=s["z"], z_scale=s["z_scale"])
            return {n: s[n] for n in ("y", "z", "z_scale") if s[n] is not None}
        B.pw_moe_ffn_backward(s["shape"], S, s["dy"], s["x"], s["w_gate_up"], s["w_down"], s["z"], s["ws"],
                              offsets=s["offsets"], act=act, z_scale=s["z_scale"], dx=s["dx"],
                              dw_gate_up=s["dw_gate_up"], dw_down=s["dw_down"])
        return {n: s[n] for n in ("dx", "dw_gate_up", "dw_down")}
    N, K = s["N"], s["K"]
    if "ws" not in s:
        size = B.pw_moe_product_workspace_bytes if op == "product" else B.pw_moe_product_backward_workspace_bytes
        s["ws"] = torch.empty(size(E, S, N, K), dtype=torch.uint8, device="cuda")
    if op == "product":
        B.pw_moe_product(E, S, N, K, s["x"], s["w"], s["y"], s["ws"], offsets=s["offsets"], bias=s["bias"], act=act,
                         residual=s["residual"], pre=s["pre"])
        return {n: s[n] for n in ("y", "pre") if s[n] is not None}
    B.pw_moe_product_backward(E, S, N, K, s["dy"], s["x"], s["w"], s["ws"], offsets=s["offsets"], act=act,
                              pre=s["pre"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"])
    return {n: s[n] for n in ("dx", "dw", "dbias") if s[n] is not None}


# ----- the definitions in 64 bits -------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    S, E = s["S"], s["E"]
    ends = [0, S] if s["offsets"] is None else s["offsets"].tolist()
    act = {"none": lambda v: v, "silu": lambda v: v / (1 + (-v).exp()),
           "gelu": lambda v: v * torch.special.ndtr(v)}[s["act"]]

    def slope(v):
        if s["act"] == "silu":
            q = 1 / (1 + (-v).exp())
            return q + v * q * (1 - q)
        if s["act"] == "gelu":
            return torch.special.ndtr(v) + v * (-v * v / 2).exp() / (2 * torch.pi) ** 0.5
        return torch.ones_like(v)

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float64, device="cuda")

    if s["op"] == "ffn":
        H, I = s["H"], s["I"]
        out = {"y": zeros(S, H)}
        if s["keep"] != "none":
            out["z"] = zeros(S, 2 * I)
        if s["keep"] == "e4m3":
            out["z_scale"] = zeros(S, 2 * -(-I // GROUP))
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            z = s["x"][at].double() @ s["w_gate_up"][e].double().T
            out["y"][at] = (act(z[:, :I]) * z[:, I:]) @ s["w_down"][e].double().T
            if s["keep"] == "same":
                out["z"][at] = z
            elif s["keep"] == "e4m3" and z.shape[0]:
                pieces = [p for half in (z[:, :I], z[:, I:]) for p in half.split(GROUP, dim=1)]
                scale = [p.abs().max(1).values.div(448).clamp(min=2.0 ** -100) for p in pieces]
                out["z_scale"][at] = torch.stack(scale, dim=1)
                out["z"][at] = torch.cat([p / v[:, None] for p, v in zip(pieces, scale)], dim=1)
        return out
    if s["op"] == "ffn_grad":
        H, I = s["H"], s["I"]
        dx, dw_gate_up, dw_down = zeros(S, H), torch.zeros_like(s["w_gate_up"], dtype=torch.float64), torch.zeros_like(s["w_down"], dtype=torch.float64)
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            x, dy = s["x"][at].double(), s["dy"][at].double()
            halves = list(s["z"][at].float().double().chunk(2, dim=1))
            if s["z_scale"] is not None:
                for i, v in enumerate(s["z_scale"][at].double().chunk(2, dim=1)):
                    halves[i] = torch.cat([p * v[:, j, None] for j, p in enumerate(halves[i].split(GROUP, dim=1))], dim=1)
            gate, up = halves
            w_gate, w_up = s["w_gate_up"][e].double().chunk(2)
            dh = dy @ s["w_down"][e].double()
            dgate, dup = dh * up * slope(gate), dh * act(gate)
            dx[at] = dgate @ w_gate + dup @ w_up
            dw_gate_up[e, :I], dw_gate_up[e, I:] = dgate.T @ x, dup.T @ x
            dw_down[e] = dy.T @ (act(gate) * up)
        return {"dx": dx, "dw_gate_up": dw_gate_up, "dw_down": dw_down}
    N, K = s["N"], s["K"]
    if s["op"] == "product":
        y, pre = zeros(S, N), zeros(S, N)
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            pre[at] = s["x"][at].double() @ s["w"][e].double().T
            if s["bias"] is not None:
                pre[at] += s["bias"][e].double()
            y[at] = act(pre[at])
            if s["residual"] is not None:
                y[at] += s["residual"][at].double()
        return {"y": y} if s["pre"] is None else {"y": y, "pre": pre}
    dx, dw, dbias = zeros(S, K), zeros(E, N, K), zeros(E, N)
    for e in range(E):
        at = slice(ends[e], ends[e + 1])
        dz = s["dy"][at].double()
        if s["pre"] is not None:
            dz = dz * slope(s["pre"][at].double())
        dx[at], dw[e], dbias[e] = dz @ s["w"][e].double(), dz.T @ s["x"][at].double(), dz.sum(0)
    return {"dx": dx, "dw": dw} if s["dbias"] is None else {"dx": dx, "dw": dw, "dbias": dbias}
