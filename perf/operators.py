"""Cases, plain forms and exact results of the FP8 block-scaled product, the
expert dispatch with its gradients, and the router's gradient.

FP8 here: OCP E4M3 codes with one fp32 scale per 128 columns of an activation
row, or per 128 x 128 block of a weight.  A block whose largest magnitude is
`amax` has b = max(amax, 2^-100), scale b/448 and codes E4M3(x * (448/b)).
"""

import math

import torch

own = False

DEV = "cuda"
B = 128                       # scale block
TINY = 2.0 ** -100            # smallest block maximum that a scale is made for


def _up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through a dense FP8 linear of the framework's dense shape: what a serving step of one request calls
        dict(name="product one token", op="product", T=1, k=1, E=0, N=2048, K=7168, skew=0.0, bad=0.0),
        # a decode batch: 256 tokens, 8 of 256 experts each, the gate and up product (8 rows an expert: the weights' bytes count)
        dict(name="product decode", op="product", T=256, k=8, E=256, N=4096, K=7168, skew=0.0, bad=0.0),
        # a prefill batch of the same layer: 65536 rows, 256 an expert
        dict(name="product prefill", op="product", T=8192, k=8, E=256, N=4096, K=7168, skew=0.0, bad=0.0),
        # few busy experts and several without rows, odd widths, a last scale block of 16 columns, some pairs without an expert
        dict(name="product ragged", op="product", T=1531, k=3, E=40, N=1001, K=1040, skew=1.2, bad=0.05),
        # a prefill batch's activations before the first product
        dict(name="quantise rows prefill", op="quantise", kind="rows", R=8192, C=7168, G=1),
        # SwiGLU and quantise between the two products of a decode batch
        dict(name="quantise swiglu decode", op="quantise", kind="swiglu", R=2048, C=2048, G=1),
        # a decode batch's rows laid out by expert
        dict(name="dispatch decode", op="dispatch", way="forward", T=256, k=8, E=256, H=7168, skew=0.0, bad=0.0),
        # gradient of the same for a training batch: each token's k row gradients summed
        dict(name="dispatch gradient", op="dispatch", way="backward", T=8192, k=8, E=256, H=7168, skew=0.0, bad=0.0),
        # gradient of the weighted sum back to tokens: of the expert rows and of the routing weights
        dict(name="combine gradient", op="combine", T=8192, k=8, E=256, H=7168, skew=0.0, bad=0.0),
        # the same for a small batch with skewed experts, a width that is no power of two, pairs without an expert
        dict(name="combine gradient small", op="combine", T=77, k=6, E=9, H=1000, skew=1.2, bad=0.1),
        # gradient of the routing weights to the router's logits for a training batch
        dict(name="router gradient", op="router", T=8192, k=8, E=256),
        # the same for few tokens and a number of experts that fills no wave
        dict(name="router gradient small", op="router", T=33, k=3, E=70),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "quantise", "dispatch", "combine", "router"])
    if op == "product":
        dense = rng.random() < 0.3
        T = _log(rng, 1, 8192)
        K = 16 * _log(rng, 4, 448)
        N = _log(rng, 32, 4096)
        if dense:
            return dict(op=op, T=T, k=1, E=0, N=N, K=K, skew=0.0, bad=0.0)
        E = _log(rng, 2, 256)
        skew = rng.choice([0.0, 0.0, 0.6, 1.2])
        if skew:                 # the plain form gives every expert the room of the busiest
            T = min(T, 1 + (1 << 31) // (E * K))
        return dict(op=op, T=T, k=rng.randint(1, min(8, E)), E=E, N=N, K=K, skew=skew, bad=rng.choice([0.0, 0.05]) if T >= 16 else 0.0)
    if op == "quantise":
        kind = rng.choice(["rows", "swiglu", "weight"])
        if kind == "weight":
            return dict(op=op, kind=kind, R=_log(rng, 1, 2048), C=16 * _log(rng, 1, 448), G=rng.randint(1, 4))
        return dict(op=op, kind=kind, R=_log(rng, 1, 8192 if kind == "rows" else 16384), C=16 * _log(rng, 1, 448 if kind == "rows" else 128), G=1)
    if op == "router":
        E = _log(rng, 3, 1024)
        return dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(2, min(8, E)), E=E)
    E = _log(rng, 2, 256)
    T = _log(rng, 1, 8192)
    c = dict(op=op, T=T, k=rng.randint(1, min(8, E)), E=E, H=8 * _log(rng, 1, 896), skew=rng.choice([0.0, 1.2]), bad=rng.choice([0.0, 0.05]) if T >= 16 else 0.0)
    if op == "dispatch":
        c["way"] = rng.choice(["forward", "backward"])
    return c


def work(case):
    c = case
    if c["op"] == "product":
        kb, nb, rows = _up(c["K"], B), _up(c["N"], B), c["T"] * c["k"]
        live = round(rows * (1 - c["bad"]))
        hit = min(max(c["E"], 1), live)      # experts with rows: about all, or one a row
        return {"bytes": c["T"] * (c["K"] + 4 * kb) + hit * (c["N"] * c["K"] + 4 * nb * kb) + 2 * live * c["N"] + 4 * rows * (c["E"] > 0),
                "flops": 2 * live * c["N"] * c["K"]}
    if c["op"] == "quantise":
        n, r = c["R"] * c["C"] * c["G"], (c["R"] if c["kind"] != "weight" else _up(c["R"], B)) * c["G"]
        return {"bytes": (4 if c["kind"] == "swiglu" else 2) * n + n + 4 * r * _up(c["C"], B), "flops": 3 * n}
    T, k = c["T"], c["k"]
    if c["op"] == "router":
        return {"bytes": 12 * T * k + 4 * T * c["E"], "flops": 4 * T * k}
    if c["op"] == "dispatch":
        return {"bytes": 2 * T * c["H"] * (1 + k) + 4 * T * k, "flops": T * k * c["H"]}
    return {"bytes": 2 * T * c["H"] * (1 + 2 * k) + 12 * T * k, "flops": 3 * T * k * c["H"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _activations(rows, cols, g):
    """bf16 activations: normal, with every 64th column 12 times as large (outlier
    channels) and rows of differing size."""
    x = torch.randn((rows, cols), generator=g, device=DEV, dtype=torch.bfloat16)
    x[:, ::64] *= 12
    return x * torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV)).to(torch.bfloat16)


def _routing(c, g):
    """k distinct experts a token (by skewed popularity), some pairs without an
    expert, and the expert order: offsets (E+1), perm (row -> pair), inverse."""
    T, k, E = c["T"], c["k"], c["E"]
    logits = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    rank = torch.argsort(torch.rand((E,), generator=g, device=DEV)).float()
    logits = logits - c["skew"] * torch.log1p(rank)
    ids = logits.topk(k, dim=1).indices.to(torch.int32)
    if c["bad"]:
        ids[torch.rand((T, k), generator=g, device=DEV) < c["bad"]] = -1
    key = torch.where(ids < 0, E, ids).reshape(-1).long()
    perm = torch.argsort(key, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    off = torch.zeros((E + 1,), dtype=torch.int64, device=DEV)
    off[1:] = counts.cumsum(0)
    return ids, off.to(torch.int32), perm.to(torch.int32), inv.to(torch.int32), int(counts.max())


def _weights(c, g):
    """E4M3 weight codes (E, N, K) and scales (E, N/128, K/128): normal 0.02
    weights whose blocks differ in size."""
    E, N, K = max(c["E"], 1), c["N"], c["K"]
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    step = max(1, (1 << 29) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        # a block's largest of 16384 normals is about 4 deviations: codes of that size with the scale drawn apart
        codes[e:e + n] = torch.randn((n, N, K), generator=g, device=DEV, dtype=torch.bfloat16).mul_(110).clamp_(-448, 448).to(torch.float8_e4m3fn)
    sf = 0.02 / 110 * torch.exp(0.3 * torch.randn((E, _up(N, B), _up(K, B)), generator=g, device=DEV))
    return codes, sf


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "product":
        s["a"], s["a_sf"] = _rows_plain(_activations(c["T"], c["K"], g))
        s["b"], s["b_sf"] = _weights(c, g)
        s["M"] = c["T"] * c["k"]
        if c["E"]:
            _, s["off"], s["perm"], _, s["most"] = _routing(c, g)
        s["out"] = torch.zeros((s["M"], c["N"]), dtype=torch.bfloat16, device=DEV)
        return s
    if c["op"] == "quantise":
        if c["kind"] == "weight":
            s["x"] = torch.randn((c["G"], c["R"], c["C"]), generator=g, device=DEV, dtype=torch.bfloat16) * 0.02
        else:
            s["x"] = _activations(c["R"], c["C"] * (2 if c["kind"] == "swiglu" else 1), g)
        return s
    if c["op"] == "router":
        T, k, E = c["T"], c["k"], c["E"]
        v, i = (2 * torch.randn((T, E), generator=g, device=DEV)).topk(k, dim=1)
        s["ids"], s["w"] = i.to(torch.int32), torch.softmax(v, dim=1)
        s["dw"] = torch.randn((T, k), generator=g, device=DEV)
        return s
    T, k, H = c["T"], c["k"], c["H"]
    _, s["off"], s["perm"], s["inv"], _ = _routing(c, g)
    if c["op"] == "dispatch":
        s["x"] = _activations(T if c["way"] == "forward" else T * k, H, g)
    else:
        s["dout"] = _activations(T, H, g)
        s["y"] = _activations(T * k, H, g)
        s["w"] = torch.softmax(torch.randn((T, k), generator=g, device=DEV), dim=1)
    return s


# ------------------------------------------------------------------ plain forms

def _pad(x, rows, cols):
    """x with its last two dimensions brought to multiples by zeros."""
    r, c = -x.shape[-2] % rows, -x.shape[-1] % cols
    return torch.nn.functional.pad(x, (0, c, 0, r)) if r or c else x


def _rows_plain(x):
    """(R, C) -> E4M3 codes (R, C) and one fp32 scale per 128 columns."""
    R, C = x.shape
    v = _pad(x.float(), 1, B).view(R, -1, B)
    b = v.abs().amax(2).clamp_min(TINY)
    return (v * (448 / b)[:, :, None]).to(torch.float8_e4m3fn).view(R, -1)[:, :C].contiguous(), b / 448


def _weight_plain(w):
    """(G, R, C) -> E4M3 codes (G, R, C) and one fp32 scale per 128 x 128."""
    G, R, C = w.shape
    v = _pad(w.float(), B, B)
    v = v.view(G, v.shape[1] // B, B, v.shape[2] // B, B)
    b = v.abs().amax((2, 4)).clamp_min(TINY)
    q = (v * (448 / b)[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(G, v.shape[1] * B, -1)[:, :R, :C].contiguous(), b / 448


def _decode_weight(q, sf):
    """E4M3 weight codes and scales -> the fp32 values they stand for, padded
    to whole blocks."""
    v = _pad(q.float(), B, B)
    G, R, C = v.shape
    v.view(G, R // B, B, C // B, B).mul_(sf[:, :, None, :, None])
    return v


def _product_plain(s):
    c = s["case"]
    K = _up(c["K"], B) * B
    a = _pad(s["a"].float(), 1, B).view(c["T"], -1, B).mul(s["a_sf"][:, :, None]).view(c["T"], K)
    w = _decode_weight(s["b"], s["b_sf"])
    if not c["E"]:
        s["out"].copy_(torch.mm(a, w[0].t())[:, :c["N"]])
        return s["out"]
    off = s["off"].long()
    d = torch.arange(s["M"], device=DEV)
    e = torch.searchsorted(off, d, right=True) - 1       # expert of each row; E behind the last
    live = e < c["E"]
    e = torch.where(live, e, 0)
    at = torch.where(live, d - off[e], s["most"])        # rows without an expert go to a spare place
    x = torch.zeros((c["E"], s["most"] + 1, K), device=DEV)
    x[e, at] = a[(s["perm"] // c["k"]).long()]
    y = torch.bmm(x, w.transpose(1, 2))[e, at, :c["N"]]
    s["out"].copy_(torch.where(live[:, None], y, s["out"].float()))
    return s["out"]


def _plain(s):
    c = s["case"]
    if c["op"] == "product":
        return _product_plain(s)
    if c["op"] == "quantise":
        if c["kind"] == "weight":
            return _weight_plain(s["x"])
        if c["kind"] == "rows":
            return _rows_plain(s["x"])
        g, u = s["x"][:, :c["C"]].float(), s["x"][:, c["C"]:].float()
        return _rows_plain(g / (1 + torch.exp(-g)) * u)
    if c["op"] == "router":
        d = s["w"] * (s["dw"] - (s["w"] * s["dw"]).sum(1, keepdim=True))
        return torch.zeros((c["T"], c["E"]), device=DEV).scatter_add_(1, s["ids"].long(), d)
    T, k, H = c["T"], c["k"], c["H"]
    inv, live = s["inv"].long(), s["inv"] < s["off"][c["E"]]
    if c["op"] == "dispatch" and c["way"] == "forward":
        rows = torch.empty((T * k, H), dtype=torch.bfloat16, device=DEV)
        rows[inv] = torch.where(live[:, None], s["x"].repeat_interleave(k, 0), 0)
        return rows
    if c["op"] == "dispatch":
        return torch.where(live[:, None], s["x"][inv].float(), 0).view(T, k, H).sum(1).to(torch.bfloat16)
    dout = s["dout"].float().repeat_interleave(k, 0)
    dy = torch.empty((T * k, H), dtype=torch.bfloat16, device=DEV)
    dy[inv] = torch.where(live[:, None], dout * s["w"].view(-1, 1), 0).to(torch.bfloat16)
    dw = torch.where(live, (dout * s["y"][inv].float()).sum(1), 0).view(T, k)
    return dy, dw


def run(state):
    s = state
    if not own:
        return _plain(s)
    import nvfp4_block_scaled_04_amd as nv
    c = s["case"]
    if c["op"] == "product":
        return nv.fp8_grouped_gemm(s["a"], s["a_sf"], s["b"], s["b_sf"], offsets=s.get("off"), M=s["M"],
                                   a_row_src=s.get("perm"), a_row_div=c["k"], out=s["out"])
    if c["op"] == "quantise":
        f = {"rows": nv.fp8_quantize, "swiglu": nv.fp8_swiglu_quantize, "weight": nv.fp8_quantize_weight}
        return f[c["kind"]](s["x"])
    if c["op"] == "router":
        return nv.router_topk_bwd(s["ids"], s["w"], s["dw"], c["E"])
    if c["op"] == "dispatch":
        f = nv.moe_dispatch if c["way"] == "forward" else nv.moe_dispatch_bwd
        return f(s["x"], s["inv"], s["off"], c["k"])
    return nv.moe_combine_bwd(s["dout"], s["y"], s["inv"], s["w"], s["off"])


# ------------------------------------------------------------------ in 64 bits

def _e4m3_64(v):
    """Nearest E4M3 value (ties to even) of float64 values up to 448 in size."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_blocks(v, dims):
    b = v.abs().amax(dims, keepdim=True).clamp_min(TINY)
    return _e4m3_64(v * 448 / b), (b / 448).squeeze(dims)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "product":
        N, K = c["N"], c["K"]
        ks = torch.arange(K, device=DEV) // B
        ns = torch.arange(N, device=DEV) // B
        out = s["out"].double()
        a = s["a"].double() * s["a_sf"].double()[:, ks]
        off = s["off"].tolist() if c["E"] else [0, c["T"]]
        for e in range(max(c["E"], 1)):
            if off[e + 1] == off[e]:
                continue
            rows = a[s["perm"][off[e]:off[e + 1]].long() // c["k"]] if c["E"] else a
            w = s["b"][e].double() * s["b_sf"][e].double()[ns][:, ks]
            out[off[e]:off[e + 1]] = rows @ w.t()
        return out
    if c["op"] == "quantise":
        x = s["x"].double()
        if c["kind"] == "swiglu":
            x = x[:, :c["C"]] * torch.sigmoid(x[:, :c["C"]]) * x[:, c["C"]:]
        if c["kind"] == "weight":
            v = _pad(x, B, B)
            q, sf = _exact_blocks(v.view(c["G"], v.shape[1] // B, B, v.shape[2] // B, B), (2, 4))
            return q.reshape(v.shape)[:, :c["R"], :c["C"]].contiguous(), sf
        v = _pad(x, 1, B)
        q, sf = _exact_blocks(v.view(c["R"], -1, B), (2,))
        return q.reshape(v.shape)[:, :c["C"]].contiguous(), sf
    if c["op"] == "router":
        w, dw = s["w"].double(), s["dw"].double()
        full = torch.zeros((c["T"], c["E"]), dtype=torch.float64, device=DEV)
        mean = (w * dw).sum(1)
        t = torch.arange(c["T"], device=DEV)
        for j in range(c["k"]):
            full[t, s["ids"][:, j].long()] = w[:, j] * (dw[:, j] - mean)
        return full
    T, k, H = c["T"], c["k"], c["H"]
    n = int(s["off"][-1])
    inv = s["inv"].long().view(T, k)
    if c["op"] == "dispatch" and c["way"] == "forward":
        rows = torch.zeros((T * k, H), dtype=torch.float64, device=DEV)
        rows[:n] = s["x"][s["perm"][:n].long() // k].double()
        return rows
    if c["op"] == "dispatch":
        dx = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        for j in range(k):
            has = inv[:, j] < n
            dx[has] += s["x"][inv[has, j]].double()
        return dx
    dy = torch.zeros((T * k, H), dtype=torch.float64, device=DEV)
    dw = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        has = inv[:, j] < n
        d = s["dout"][has].double()
        dy[inv[has, j]] = d * s["w"][has, j].double()[:, None]
        dw[has, j] = (d * s["y"][inv[has, j]].double()).sum(1)
    return dy, dw
