"""Cases, plain forms and exact results of the RMS norm (residual added, BF16 or
FP8 outputs, gradient) and of the expert layer for a few tokens.

FP8 here: OCP E4M3 codes with one fp32 scale per 128 columns of an activation
row, or per 128 x 128 block of a weight.  NVFP4: E2M1 codes, two a byte, one
E4M3 scale per 16 along K and one fp32 global scale an expert (value = code *
scale / global), in tiles of 512 rows x 128 columns.
"""

import math

import torch

own = False

DEV = "cuda"
B = 128                       # FP8 scale block; K elements of an NVFP4 tile
TINY = 2.0 ** -100            # smallest block maximum that an FP8 scale is made for
PACK = 512                    # rows of an NVFP4 tile
EPS = 1e-6


def _up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token between attention and the experts: residual added, FP8 for the products, BF16 for the router
        dict(name="norm one token", op="norm", T=1, H=7168, res=True, out="both", wide=False),
        # the same for a prefill batch
        dict(name="norm prefill", op="norm", T=8192, H=7168, res=True, out="both", wide=False),
        # queries and keys normalised head by head: many short rows
        dict(name="norm heads", op="norm", T=65536, H=128, res=False, out="bf16", wide=True),
        # a batch of odd size, a last scale block of 16 columns, FP8 only
        dict(name="norm ragged", op="norm", T=777, H=1040, res=True, out="fp8", wide=True),
        # gradient of the norm for a training batch, with the residual branch's gradient added
        dict(name="norm gradient", op="grad", T=8192, H=7168, res=True, wide=False),
        # the same for few rows of an odd width, no residual branch
        dict(name="norm gradient small", op="grad", T=77, H=1000, res=False, wide=True),
        # one request's serving step through a large FP8 expert layer: 8 of 256 experts, the weights' bytes count
        dict(name="experts fp8 one token", op="experts", fmt="fp8", T=1, H=7168, I=2048, E=256, k=8, skew=0.0, bad=0.0),
        # the same layer in NVFP4
        dict(name="experts nvfp4 one token", op="experts", fmt="nvfp4", T=1, H=7168, I=2048, E=256, k=8, skew=0.0, bad=0.0),
        # sixteen requests' step: about a hundred experts, one or two tokens each
        dict(name="experts nvfp4 batch", op="experts", fmt="nvfp4", T=16, H=7168, I=2048, E=256, k=8, skew=0.0, bad=0.0),
        # a small layer, where launches and latency count
        dict(name="experts fp8 small", op="experts", fmt="fp8", T=4, H=2048, I=768, E=128, k=8, skew=0.0, bad=0.0),
        # few busy experts, odd widths, pairs without an expert
        dict(name="experts fp8 ragged", op="experts", fmt="fp8", T=13, H=1040, I=528, E=40, k=3, skew=1.2, bad=0.1),
        # a small NVFP4 layer for one token
        dict(name="experts nvfp4 small", op="experts", fmt="nvfp4", T=1, H=2048, I=768, E=32, k=4, skew=0.0, bad=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "grad", "experts", "experts", "experts"])
    if op != "experts":
        T, wide, res = _log(rng, 1, 8192), rng.random() < 0.5, rng.random() < 0.6
        if op == "grad":
            return dict(op=op, T=T, H=8 * _log(rng, 2, 896), res=res, wide=wide)
        out = rng.choice(["bf16", "fp8", "both"])
        return dict(op=op, T=T, H=8 * _log(rng, 2, 896) if out == "bf16" else 16 * _log(rng, 1, 448), res=res, out=out, wide=wide)
    fmt = rng.choice(["fp8", "nvfp4"])
    step, E, T = 16 if fmt == "fp8" else 128, _log(rng, 2, 256), rng.randint(1, 16)
    return dict(op=op, fmt=fmt, T=T, H=step * _log(rng, 1, 7168 // step), I=step * _log(rng, 1, 2048 // step), E=E,
                k=rng.randint(1, min(8, E)), skew=rng.choice([0.0, 0.0, 1.2]), bad=rng.choice([0.0, 0.1]) if T >= 4 else 0.0)


def work(case):
    c = case
    if c["op"] == "norm":
        n, r = c["T"] * c["H"], c["res"]
        o = {"bf16": 2 * n, "fp8": n + 4 * c["T"] * _up(c["H"], B)}
        out = sum(o.values()) if c["out"] == "both" else o[c["out"]]
        return {"bytes": 2 * n + (4 * n if r else 0) + out + (4 if c["wide"] else 2) * c["H"], "flops": 6 * n}
    if c["op"] == "grad":
        n = c["T"] * c["H"]
        return {"bytes": 6 * n + (2 * n if c["res"] else 0) + 4 * c["T"] + (8 if c["wide"] else 6) * c["H"], "flops": 10 * n}
    T, H, I, E, k = (c[i] for i in "THIEk")
    live = T * k * (1 - c["bad"])
    hit = E * (1 - (1 - k / E) ** T) if not c["skew"] else min(E, live) / 2      # experts with a token, about
    per = 3 * H * I + 4 * (_up(2 * I, B) * _up(H, B) + _up(H, B) * _up(I, B)) if c["fmt"] == "fp8" else 3 * H * I * 9 / 16
    return {"bytes": int(hit * per) + 4 * T * H + 8 * T * k, "flops": int(6 * live * H * I)}


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


def _ids(c, g):
    """k distinct experts a token (by skewed popularity), some pairs without one."""
    T, k, E = c["T"], c["k"], c["E"]
    logits = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    rank = torch.argsort(torch.rand((E,), generator=g, device=DEV)).float()
    v, ids = (logits - c["skew"] * torch.log1p(rank)).topk(k, dim=1)
    ids = ids.to(torch.int32)
    if c["bad"]:
        ids[torch.rand((T, k), generator=g, device=DEV) < c["bad"]] = -1
    return ids, torch.softmax(v, dim=1)


def _fp8_weight(E, N, K, g):
    """E4M3 codes (E, N, K) and scales (E, N/128, K/128): normal weights of
    deviation 0.02 whose blocks differ in size."""
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    step = max(1, (1 << 29) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        codes[e:e + n] = torch.randn((n, N, K), generator=g, device=DEV, dtype=torch.bfloat16).mul_(110).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return codes, 0.02 / 110 * torch.exp(0.3 * torch.randn((E, _up(N, B), _up(K, B)), generator=g, device=DEV))


def _nvfp4_weight(E, N, K, g):
    """Packed NVFP4 weights: codes (E, N/512, K/128, 512, 64), scales (..., 8),
    both flat and zero behind row N, and a global scale an expert.  Codes are
    drawn evenly (deviation 3.1), scales between 2^6 and 2^8, global scales so
    that values deviate by about 0.02."""
    tiles = _up(N, PACK)
    q = torch.randint(0, 256, (E, tiles, K // B, PACK, 64), generator=g, device=DEV, dtype=torch.uint8)
    sf = torch.randint(104, 121, (E, tiles, K // B, PACK, 8), generator=g, device=DEV, dtype=torch.uint8)
    if N % PACK:
        q[:, -1, :, N % PACK:] = 0
        sf[:, -1, :, N % PACK:] = 0
    gs = 2e4 * torch.exp(0.3 * torch.randn((E,), generator=g, device=DEV))
    return q.flatten(), sf.flatten(), gs


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    T, H = c["T"], c["H"]
    if c["op"] != "experts":
        w = 1 + 0.2 * torch.randn((H,), generator=g, device=DEV)
        s["w"] = w if c["wide"] else w.to(torch.bfloat16)
        s["x"] = _activations(T, H, g)
        if c["op"] == "norm":
            s["res"] = _activations(T, H, g) if c["res"] else None
        else:                      # x is what the forward pass stored, with its 1/rms
            s["dy"] = _activations(T, H, g)
            s["dh"] = _activations(T, H, g) if c["res"] else None
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
        return s
    s["x"] = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    s["ids"], s["w"] = _ids(c, g)
    make = _fp8_weight if c["fmt"] == "fp8" else _nvfp4_weight
    s["w1"], s["w2"] = make(c["E"], 2 * c["I"], H, g), make(c["E"], H, c["I"], g)
    return s


# ------------------------------------------------------------------ plain forms

def _pad(x, rows, cols):
    """x with its last two dimensions brought to multiples by zeros."""
    r, c = -x.shape[-2] % rows, -x.shape[-1] % cols
    return torch.nn.functional.pad(x, (0, c, 0, r)) if r or c else x


def _rows_plain(v):
    """fp32 (R, C) -> E4M3 codes (R, C) and one fp32 scale per 128 columns."""
    R, C = v.shape
    v = _pad(v, 1, B).view(R, -1, B)
    b = v.abs().amax(2).clamp_min(TINY)
    return (v * (448 / b)[:, :, None]).to(torch.float8_e4m3fn).view(R, -1)[:, :C].contiguous(), b / 448


def _norm_plain(s):
    c = s["case"]
    h = s["x"]
    if s["res"] is not None:
        h = (h.float() + s["res"].float()).to(torch.bfloat16)
    f = h.float()
    v = f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    out = {"h": h} if s["res"] is not None else {}
    if c["out"] != "bf16":
        out["q"], out["sf"] = _rows_plain(v)
    if c["out"] != "fp8":
        out["y"] = v.to(torch.bfloat16)
    return out


def _grad_plain(s):
    n = s["x"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - n * (g * n).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * n).sum(0)}


def _e2m1(dtype):
    return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=DEV)


def _decode(c, w, e, N, K, dtype):
    """Weights of the experts e as (len(e), N, K) values."""
    n = e.numel()
    if c["fmt"] == "fp8":
        q, sf = w
        v = _pad(q.view(torch.uint8).index_select(0, e).view(torch.float8_e4m3fn).to(dtype), B, B)
        v.view(n, v.shape[1] // B, B, -1, B).mul_(sf.index_select(0, e).to(dtype)[:, :, None, :, None])
        return v[:, :N, :K]
    q, sf, gs = w
    tiles, S = _up(N, PACK), K // B
    q = q.view(-1, tiles * S * PACK * 64).index_select(0, e).long()
    v = _e2m1(dtype)[torch.stack((q & 15, q >> 4), -1)].view(n, tiles, S, PACK, 8, 16)
    sf = sf.view(-1, tiles * S * PACK * 8).index_select(0, e).view(torch.float8_e4m3fn).to(dtype)
    v = (v * sf.view(n, tiles, S, PACK, 8, 1)).view(n, tiles, S, PACK, B).transpose(2, 3)
    return v.reshape(n, tiles * PACK, K)[:, :N] / gs.index_select(0, e).to(dtype)[:, None, None]


def _gate_up(c, a):
    """Gate and up columns of the first product: halves, or (NVFP4) interleaved at 8."""
    if c["fmt"] == "fp8":
        return a[..., :c["I"]], a[..., c["I"]:]
    a = a.view(*a.shape[:-1], -1, 2, 8)
    return a[..., 0, :].flatten(-2), a[..., 1, :].flatten(-2)


def _experts(s, dtype):
    c = s["case"]
    T, H, I, E, k = (c[i] for i in "THIEk")
    ids = s["ids"].flatten().long()
    live = (ids >= 0) & (ids < E)
    ids, w = torch.where(live, ids, 0), torch.where(live, s["w"].flatten(), 0).to(dtype)
    x, y = s["x"].to(dtype).repeat_interleave(k, 0), []
    for i in range(0, T * k, 4):            # four pairs at a time: what their decoded weights take
        e = ids[i:i + 4]
        a = torch.bmm(_decode(c, s["w1"], e, 2 * I, H, dtype), x[i:i + 4, :, None])[..., 0]
        g, u = _gate_up(c, a)
        h = g / (1 + torch.exp(-g)) * u
        y.append(torch.bmm(_decode(c, s["w2"], e, H, I, dtype), h[..., None])[..., 0] * w[i:i + 4, None])
    return torch.cat(y).view(T, k, H).sum(1)


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _norm_plain(s)
    if op == "grad":
        return _grad_plain(s)
    return _experts(s, torch.float32).to(torch.bfloat16)


def run(state):
    s = state
    if not own:
        return _plain(s)
    import nvfp4_block_scaled_04_amd as nv
    c = s["case"]
    if c["op"] == "norm":
        if c["out"] == "bf16":
            y, h, _ = nv.rmsnorm(s["x"], s["w"], residual=s["res"], eps=EPS)
            out = {"y": y}
        else:
            q, sf, y, h, _ = nv.fp8_rmsnorm(s["x"], s["w"], residual=s["res"], eps=EPS, need_y=c["out"] == "both")
            out = {"q": q, "sf": sf}
            if y is not None:
                out["y"] = y
        return {"h": h, **out} if c["res"] else out
    if c["op"] == "grad":
        dx, dw = nv.rmsnorm_bwd(s["dy"], s["x"], s["w"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if c["fmt"] == "fp8":
        return nv.moe_expert_forward_few_fp8(s["x"], s["ids"], s["w"], *s["w1"], *s["w2"])
    (q1, s1, g1), (q2, s2, g2) = s["w1"], s["w2"]
    w = nv.ExpertWeights(nv.PackedWeight(q1, s1, c["E"], 2 * c["I"], c["H"]), g1, nv.PackedWeight(q2, s2, c["E"], c["H"], c["I"]), g2)
    return nv.moe_expert_forward_few(s["x"], s["ids"], s["w"], w)


# ------------------------------------------------------------------ in 64 bits

def _e4m3_64(v):
    """Nearest E4M3 value (ties to even) of float64 values up to 448 in size."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_norm(s):
    c = s["case"]
    h = s["x"].double()
    out = {}
    if s["res"] is not None:
        out["h"] = h + s["res"].double()
        h = out["h"].to(torch.bfloat16).double()         # the norm is of the stored sum
    v = h / torch.sqrt((h * h).sum(1, keepdim=True) / c["H"] + EPS) * s["w"].double()
    if c["out"] != "bf16":
        p = torch.nn.functional.pad(v, (0, -c["H"] % B)).view(c["T"], -1, B)
        b = p.abs().amax(2, keepdim=True).clamp_min(TINY)
        out["q"], out["sf"] = _e4m3_64(p * 448 / b).view(c["T"], -1)[:, :c["H"]].contiguous(), (b / 448)[..., 0]
    if c["out"] != "fp8":
        out["y"] = v
    return out


def _exact_grad(s):
    """dx by the chain rule through 1/rms, dw as the sum over rows."""
    x, r, dy, w = s["x"].double(), s["rstd"].double()[:, None], s["dy"].double(), s["w"].double()
    dr = (dy * w * x).sum(1, keepdim=True)               # gradient of 1/rms
    dx = dy * w * r - dr * r ** 3 * x / x.shape[1]
    if s["dh"] is not None:
        dx += s["dh"].double()
    return {"dx": dx, "dw": (dy * x * r).sum(0)}


def _exact_experts(s):
    """Expert by expert over its tokens, weights decoded element by element."""
    c = s["case"]
    T, H, I, E, k = (c[i] for i in "THIEk")
    ids = s["ids"].tolist()
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)

    def weight(w, e, N, K):
        n, kk = torch.arange(N, device=DEV)[:, None], torch.arange(K, device=DEV)[None]
        if c["fmt"] == "fp8":
            return w[0][e].double() * w[1][e].double()[n // B, kk // B]
        tiles, S = _up(N, PACK), K // B
        at = ((e * tiles + n // PACK) * S + kk // B) * PACK + n % PACK          # row of a stage
        code = (w[0][at * 64 + kk % B // 2] >> (4 * (kk % 2)).to(torch.uint8)) & 15
        b = w[1][at * 8 + kk % B // 16].long()
        mant, ex = (b & 7).double(), (b >> 3) & 15
        scale = torch.where(ex == 0, mant * 2.0 ** -9, (1 + mant / 8) * torch.exp2(ex.double() - 7))
        return _e2m1(torch.float64)[code.long()] * scale / w[2][e].double()

    for e in sorted({i for row in ids for i in row if 0 <= i < E}):
        pairs = [(t, j) for t in range(T) for j in range(k) if ids[t][j] == e]
        t, j = (torch.tensor(v, device=DEV) for v in zip(*pairs))
        a = s["x"][t].double() @ weight(s["w1"], e, 2 * I, H).t()
        g, u = _gate_up(c, a)
        y = (g * torch.sigmoid(g) * u) @ weight(s["w2"], e, H, I).t()
        out.index_add_(0, t, y * s["w"][t, j].double()[:, None])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    return _exact_grad(s) if case["op"] == "grad" else _exact_experts(s)
