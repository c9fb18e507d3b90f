"""The training and position operators next to block-sparse video attention, as
cases that can be timed and compared: rotary positions over three axes, the
per-head norm of queries and keys with that rotation in the same pass, its
gradients, and the gradients of block-sparse attention.

A case names a kind and its sizes; `prepare` draws its inputs, `run` computes
it in plain torch operations (or, with `own`, through the library's entry
points), `exact` gives the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

#: the token grid of the headline workload
WAN = {"T": 21, "Hg": 30, "Wg": 52}


# ------------------------------------------------------------------ cases
def _rope(name, kind, B, Hq, Hk, d, T, Hg, Wg, dims, layout, dtype, perm, tail=0, values=False, head_weights=False,
          start=0, strided=True):
    return {"name": name, "kind": kind, "B": B, "Hq": Hq, "Hk": Hk, "d": d, "T": T, "Hg": Hg, "Wg": Wg,
            "dt": dims[0], "dh": dims[1], "dw": dims[2], "layout": layout, "dtype": dtype, "perm": perm, "tail": tail,
            "values": values, "head_weights": head_weights, "start": start, "strided": strided}


def _attend(name, B, H, N, d, block, dtype, scope, keep):
    return {"name": name, "kind": "attend_grad", "B": B, "H": H, "N": N, "d": d, "block": block, "dtype": dtype,
            "scope": scope, "keep": keep}


def listed():
    return [
        # one new token of a streamed clip, far into it: the rotation's latency
        _rope("rope_new_token", "rope", 1, 12, 12, 128, 1, 1, 1, (44, 42, 42), "interleaved", "bf16", "none", start=4001),
        # a video layer's queries and keys, rotated on their way into 3D block order
        _rope("rope_video", "rope", 1, 12, 12, 128, **WAN, dims=(44, 42, 42), layout="interleaved", dtype="bf16", perm="tiles"),
        # images with two axes, half-split pairs, odd width, fp32
        _rope("rope_image_f32", "rope", 2, 8, 8, 64, 1, 45, 77, (0, 32, 32), "half", "f32", "none"),
        # one frame followed by text tokens that take no rotation; shared key heads; part of the head rotated
        _rope("norm_rope_frame", "norm_rope", 1, 24, 6, 128, 1, 30, 52, (32, 32, 32), "half", "bf16", "none", tail=77),
        # the whole front end of a video layer: norm and rotate q and k, put q, k, v into 3D block order
        _rope("norm_rope_video", "norm_rope", 1, 12, 12, 128, **WAN, dims=(44, 42, 42), layout="interleaved", dtype="bf16",
              perm="tiles", values=True),
        # its gradients on a small odd grid in fp32, a weight row for each head
        _rope("norm_rope_grad_small_f32", "norm_rope_grad", 2, 3, 3, 64, 3, 7, 31, (20, 22, 22), "interleaved", "f32",
              "tiles", head_weights=True, strided=False),
        # its gradients for the video layer
        _rope("norm_rope_grad_video", "norm_rope_grad", 1, 12, 12, 128, **WAN, dims=(44, 42, 42), layout="interleaved",
              dtype="bf16", perm="tiles", values=True),
        # attention's gradients on the smallest workload: latency, fp32
        _attend("attend_grad_tiny_f32", 1, 2, 256, 64, 64, "f32", "row", 0.6),
        # 128-token blocks, a ragged last one, query blocks that keep nothing
        _attend("attend_grad_ragged_b128", 2, 6, 4884, 64, 128, "bf16", "head", 0.35),
        # every query token with its own blocks
        _attend("attend_grad_tokens", 1, 4, 3120, 128, 64, "bf16", "token", 0.25),
        # the video layer at the share of blocks that reaches 99 % of the mass
        _attend("attend_grad_video", 1, 12, 32760, 128, 64, "bf16", "row", 0.9),
        # the video layer at the share that a cheap score keeps
        _attend("attend_grad_video_sparse", 1, 12, 32760, 128, 64, "bf16", "head", 0.25),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rope", "norm_rope", "norm_rope_grad", "attend_grad", "attend_grad"])
    if kind == "attend_grad":
        d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "bf16", "f32"])
        scope = rng.choice(["row", "head", "token"])
        block = 64 if scope == "token" else rng.choice([64, 128])
        B, H = rng.choice([1, 1, 2]), _log(rng, 1, 12)
        # fp32 layers and per-token lists are the small workloads here
        N = _log(rng, 130, 2600 if dtype == "f32" else 6000 if scope == "token" else 20000)
        c = _attend("", B, H, N, d, block, dtype, scope, round(rng.uniform(0.1, 0.9), 3))
    else:
        d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "f32"])
        layout = rng.choice(["interleaved", "half"])
        if layout == "interleaved":
            dt = 2 * rng.randint(0, d // 8)
            dh = 2 * rng.randint(1, d // 6)
            dims = (dt, dh, min(dh, d - dt - dh))
        else:
            dims = rng.choice([(0, d // 2, d // 2), (d // 4, d // 4, d // 4), (d // 4, 3 * d // 8, 3 * d // 8)])
        T, Hg, Wg = _log(rng, 1, 21), _log(rng, 1, 30), _log(rng, 1, 52)
        Hk = _log(rng, 1, 8)
        Hq = Hk * rng.choice([1, 1, 2])
        c = _rope("", kind, rng.choice([1, 1, 2]), Hq, Hk, d, T, Hg, Wg, dims, layout, dtype, rng.choice(["none", "tiles", "random"]),
                  tail=rng.choice([0, 0, _log(rng, 1, 300)]), values=kind != "rope" and rng.random() < 0.5,
                  head_weights=kind != "rope" and rng.random() < 0.3, start=rng.choice([0, _log(rng, 1, 5000)]),
                  strided=rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _grid(case):
    return case["T"], case["Hg"], case["Wg"]


def _dims(case):
    return case["dt"], case["dh"], case["dw"]


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _angle_rows(case):
    """Angles [rows of the table] in 64 bits: for each axis, position x (half of its dims) frequencies."""
    parts = []
    for extent, dim, first in zip(_grid(case), _dims(case), (case["start"], 0, 0)):
        freq = 10000.0 ** (-2.0 * torch.arange(dim // 2, device="cuda", dtype=torch.float64) / max(dim, 1))
        pos = torch.arange(first, first + extent, device="cuda", dtype=torch.float64)
        parts.append((pos[:, None] * freq).reshape(-1))
    return torch.cat(parts)


def _rope_order(case, gen):
    """Source token of each slot, int32, or None."""
    T, Hg, Wg = _grid(case)
    n = T * Hg * Wg + case["tail"]
    if case["perm"] == "none":
        return None
    if case["perm"] == "random":
        return torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
    tok = torch.arange(n, device="cuda")
    t, h, w = tok // (Hg * Wg), tok // Wg % Hg, tok % Wg          # 4 x 4 x 4 tiles, raster order within a tile
    tile = (t // 4 * (-(-Hg // 4)) + h // 4) * (-(-Wg // 4)) + w // 4
    tile[T * Hg * Wg:] = 2 ** 40                                  # tokens past the grid stay last
    return torch.argsort(tile, stable=True).to(torch.int32)


def _prepare_rope(case, gen):
    T, Hg, Wg = _grid(case)
    B, n, d, dtype = case["B"], T * Hg * Wg + case["tail"], case["d"], _dtype(case)
    heads = [case["Hq"], case["Hk"]] + ([case["Hk"]] if case["values"] else [])

    def rows(H, spread):
        x = (_normal(gen, B, n, H, d) * spread).to(dtype)         # as a projection leaves it
        return x.transpose(1, 2) if case["strided"] else x.transpose(1, 2).contiguous()
    angle = _angle_rows(case)
    s = {"case": case, "xs": [rows(H, sp) for H, sp in zip(heads, (1.5, 0.8, 1.0))], "perm": _rope_order(case, gen),
         "table": torch.stack([angle.cos(), angle.sin()], -1).float(), "grid": _grid(case), "dims": _dims(case)}
    if case["kind"] != "rope":
        s["weights"] = [1 + 0.2 * _normal(gen, *((H, d) if case["head_weights"] else (d,))) for H in heads[:2]]
        s["weights"] += [None] * (len(heads) - 2)
    if case["kind"] == "norm_rope_grad":
        s["dys"] = [torch.empty_like(x).copy_(_normal(gen, *x.shape)) for x in s["xs"]]
    return s


def _kept(case, gen):
    """Truth values [B, H, rows, nB]: which key blocks each query block (scope
    "token": each query token) keeps: near ones first, with noise, as many as
    the share says in the mean; some rows keep none in the scopes where that
    can happen."""
    B, H, N, block, scope = case["B"], case["H"], case["N"], case["block"], case["scope"]
    nB = -(-N // block)
    rows = N if scope == "token" else nB
    at = torch.arange(rows, device="cuda") // (block if scope == "token" else 1)
    near = (at[:, None] - torch.arange(nB, device="cuda")).abs() / nB
    score = torch.rand(B, H, rows, nB, generator=gen, device="cuda") * 0.7 - near
    if scope == "head":
        level = torch.quantile(score.reshape(B, H, -1)[..., :: max(1, nB * nB // 65536)], 1 - case["keep"], dim=-1)
        keep = score >= level[..., None, None]
    else:
        spread = 2 * min(0.5, 1 / case["keep"] - 1)
        share = case["keep"] * (1 + spread * (torch.rand(B, H, rows, 1, generator=gen, device="cuda") - 0.5))
        keep = score.argsort(-1, descending=True).argsort(-1) < (share * nB).ceil()
    if scope != "row" and rows > 2:
        keep[:, :, torch.randint(rows, (1 + rows // 50,), generator=gen, device="cuda")] = False
        keep[:, :, 0, 0] = True                                   # a head keeps one pair at least
    return keep


def _pairs(case, keep, b, h):
    """The kept (query, key) pairs of one head, truth values [N, N]."""
    keep = keep[b, h].repeat_interleave(case["block"], 1)[:, :case["N"]]
    return keep if case["scope"] == "token" else keep.repeat_interleave(case["block"], 0)[:case["N"]]


def _prepare_attend(case, gen):
    B, H, N, d, dtype = case["B"], case["H"], case["N"], case["d"], _dtype(case)
    place = torch.linspace(0, 6.0, N, device="cuda")[:, None] * (2.0 ** torch.arange(0, 4, device="cuda"))
    wave = torch.cat([place.cos(), place.sin()], 1)               # near tokens look alike
    base = torch.einsum("nf,hfd->hnd", wave, _normal(gen, H, 8, d)) * 0.35
    q, k = ((base + 0.6 * _normal(gen, B, H, N, d)).to(dtype) for _ in range(2))
    v, dout = (_normal(gen, B, H, N, d).to(dtype) for _ in range(2))
    keep = _kept(case, gen)
    out, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    for b in range(B):                                            # one head's pairs at a time
        for h in range(H):
            z = (q[b, h].float() @ k[b, h].float().T).mul_(d ** -0.5).masked_fill_(~_pairs(case, keep, b, h), -math.inf)
            lse[b, h] = torch.logsumexp(z, 1)
            out[b, h] = z.sub_(lse[b, h].nan_to_num(neginf=0.0)[:, None]).exp_() @ v[b, h].float()
    s = {"case": case, "q": q, "k": k, "v": v, "dout": dout, "out": out, "lse": lse, "keep": keep}
    if own:
        # the frozen block list that a program keeps for many steps
        import block_sparse_attention_16_b200 as lbsa
        if case["scope"] == "token":
            s["blocks"] = lbsa.lbsa_select_tokens(keep.float().mul_(0.5), case["block"], 1 - 2.0 ** -24)
        else:
            nB = keep.shape[-1]
            words = torch.nn.functional.pad(keep, (0, -nB % 32)).view(B, H, nB, -1, 32).long()
            words = (words << torch.arange(32, device="cuda")).sum(-1)
            s["blocks"] = lbsa.lbsa_blockset_from_bitmask(torch.where(words < 2 ** 31, words, words - 2 ** 32).int(),
                                                          case["block"])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_attend(case, gen) if case["kind"] == "attend_grad" else _prepare_rope(case, gen)


# ------------------------------------------------------------------ one pass
def _turns(s):
    """cos and sin [N, rotated dims / 2] of every source token in fp32."""
    (T, Hg, Wg), (dt, dh, dw) = s["grid"], s["dims"]
    axes = s["table"].split([T * dt // 2, Hg * dh // 2, Wg * dw // 2])
    tok = torch.arange(T * Hg * Wg, device="cuda")
    rows = torch.cat([axes[0].view(T, -1, 2)[tok // (Hg * Wg)], axes[1].view(Hg, -1, 2)[tok // Wg % Hg],
                      axes[2].view(Wg, -1, 2)[tok % Wg]], 1)
    still = torch.tensor([1.0, 0.0], device="cuda").expand(s["case"]["tail"], rows.shape[1], 2)
    return torch.cat([rows, still]).unbind(-1)


def _rotate(x, cos, sin, layout):
    rd = 2 * cos.shape[-1]
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if layout == "interleaved" else (x[..., :rd // 2], x[..., rd // 2:rd])
    y = x.clone()
    if layout == "interleaved":
        y[..., 0:rd:2], y[..., 1:rd:2] = a * cos - b * sin, a * sin + b * cos
    else:
        y[..., :rd // 2], y[..., rd // 2:rd] = a * cos - b * sin, a * sin + b * cos
    return y


def _scaled(x, w):
    """x / rms(x), and the same times the weight."""
    n = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    return n, n * (w if w.dim() == 1 else w[:, None])


def _plain_rope(s):
    cos, sin = _turns(s)
    layout, outs = s["case"]["layout"], []
    for x, w in zip(s["xs"], s.get("weights", (None, None))):
        y = x.float()
        if w is not None:
            y = _scaled(y, w)[1]
        if w is not None or "weights" not in s:
            y = _rotate(y, cos, sin, layout)
        outs.append((y if s["perm"] is None else y[:, :, s["perm"].long()]).to(x.dtype))
    return outs


def _plain_rope_grad(s):
    cos, sin = _turns(s)
    layout, dxs, dws = s["case"]["layout"], [], []
    for x, dy, w in zip(s["xs"], s["dys"], s["weights"]):
        g = dy.float()
        if s["perm"] is not None:
            g = torch.empty_like(g).index_copy_(2, s["perm"].long(), g)
        if w is not None:
            g, x32 = _rotate(g, cos, -sin, layout), x.float()
            n = _scaled(x32, w)[0]
            dws.append((g.double() * n).sum((0, 2) if w.dim() == 2 else (0, 1, 2)).float())
            g = g * (w if w.dim() == 1 else w[:, None])
            g = (g - n * (g * n).mean(-1, keepdim=True)) * (x32.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        dxs.append(g.to(x.dtype))
    return dxs, dws


def _plain_attend_grad(s):
    case, scale = s["case"], s["case"]["d"] ** -0.5
    dq, dk, dv = (torch.empty_like(s["q"]) for _ in range(3))
    for b in range(case["B"]):                                    # one head's pairs at a time fit the card
        for h in range(case["H"]):
            q, k, v, do = (s[x][b, h].float() for x in ("q", "k", "v", "dout"))
            p = (q @ k.T).mul_(scale).masked_fill_(~_pairs(case, s["keep"], b, h), -math.inf)
            p = p.sub_(s["lse"][b, h].nan_to_num(neginf=0.0)[:, None]).exp_()
            dv[b, h] = p.T @ do
            dp = do @ v.T
            ds = p.mul_(dp.sub_((p * dp).sum(1, keepdim=True)))
            dq[b, h] = (ds @ k).mul_(scale)
            dk[b, h] = (ds.T @ q).mul_(scale)
    return dq, dk, dv


def run(s):
    kind = s["case"]["kind"]
    if not own:
        return {"rope": _plain_rope, "norm_rope": _plain_rope, "norm_rope_grad": _plain_rope_grad,
                "attend_grad": _plain_attend_grad}[kind](s)
    import block_sparse_attention_16_b200 as lbsa
    if kind == "attend_grad":
        return lbsa.lbsa_attend_backward(s["q"], s["k"], s["v"], s["blocks"], s["out"], s["lse"], s["dout"])
    pos = {"table": s["table"], "grid": s["grid"], "dims": s["dims"], "perm": s["perm"], "layout": s["case"]["layout"]}
    if kind == "rope":
        return lbsa.lbsa_rope(s["xs"], **pos)
    if kind == "norm_rope":
        return lbsa.lbsa_norm_rope(s["xs"], s["weights"], **pos)
    dxs, dws = lbsa.lbsa_norm_rope_backward(s["dys"], s["xs"], s["weights"], **pos)
    return dxs, [w for w in dws if w is not None]


# ------------------------------------------------------------------ what it takes
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "attend_grad":
        B, H, N, d = (case[x] for x in ("B", "H", "N", "d"))
        nB = -(-N // case["block"])
        listed_bytes = B * H * nB * nB * case["keep"] * (12 if case["scope"] == "token" else 4)
        # q, k, v, out, dout in and dq, dk, dv out; five products over the kept pairs
        return {"bytes": 8 * B * H * N * d * es + 4 * B * H * N + listed_bytes,
                "flops": 10 * d * case["keep"] * B * H * float(N) * N}
    T, Hg, Wg = _grid(case)
    n = T * Hg * Wg + case["tail"]
    turned = case["B"] * n * (case["Hq"] + case["Hk"]) * case["d"]
    rows = turned + (case["B"] * n * case["Hk"] * case["d"] if case["values"] else 0)
    table = 4 * (T * case["dt"] + Hg * case["dh"] + Wg * case["dw"]) + (4 * n if case["perm"] != "none" else 0)
    if case["kind"] == "norm_rope_grad":
        return {"bytes": es * (2 * rows + turned) + table, "flops": 16 * turned}
    return {"bytes": 2 * es * rows + table, "flops": (3 if case["kind"] == "rope" else 7) * turned}


# ------------------------------------------------------------------ in 64 bits
def _turn_exact(case, x):
    """x [B, H, N, d] in 64 bits with each pair, as a complex number, turned by its angle."""
    T, Hg, Wg = _grid(case)
    tok = torch.arange(T * Hg * Wg, device="cuda")
    pos = (tok // (Hg * Wg) + case["start"], tok // Wg % Hg, tok % Wg)
    angle = torch.cat([p.double()[:, None] * torch.exp(-math.log(10000.0) * 2 * torch.arange(m // 2, device="cuda").double() / m)
                       for p, m in zip(pos, _dims(case)) if m], 1)
    angle = torch.nn.functional.pad(angle, (0, 0, 0, case["tail"]))
    rd = 2 * angle.shape[1]
    head = x[..., :rd]
    pair = head.unflatten(-1, (-1, 2)) if case["layout"] == "interleaved" else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(angle), angle))
    turned = turned if case["layout"] == "interleaved" else turned.transpose(-1, -2)
    return torch.cat([turned.flatten(-2), x[..., rd:]], -1)


def _front_exact(case, x, w, turn, perm):
    if w is not None:
        x = torch.nn.functional.normalize(x, dim=-1, eps=0.0) * math.sqrt(case["d"]) \
            * (x.square().mean(-1, keepdim=True) / (x.square().mean(-1, keepdim=True) + 1e-6)).sqrt()
        x = x * w.reshape((1, -1, 1, case["d"]))
    if turn:
        x = _turn_exact(case, x)
    return x if perm is None else x.index_select(2, perm.long())


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] != "attend_grad":
        weights = s.get("weights", [None] * len(s["xs"]))
        outs, dxs, dws = [], [], []
        for i, (x, w) in enumerate(zip(s["xs"], weights)):
            x = x.double().requires_grad_()
            w = None if w is None else w.double().requires_grad_()
            y = _front_exact(case, x, w, i < 2, s["perm"])
            outs.append(y.detach())
            if case["kind"] == "norm_rope_grad":
                got = torch.autograd.grad(y, [x] if w is None else [x, w], s["dys"][i].double())
                dxs.append(got[0])
                dws += list(got[1:])
        return (dxs, dws) if case["kind"] == "norm_rope_grad" else outs
    grads = [torch.empty(s["q"].shape, dtype=torch.float64, device="cuda") for _ in range(3)]
    step = max(256, 2 ** 28 // case["N"])                         # query rows at a time
    for b in range(case["B"]):
        for h in range(case["H"]):
            q, k, v = (s[x][b, h].double().requires_grad_() for x in ("q", "k", "v"))
            total = [torch.zeros_like(k), torch.zeros_like(v)]
            for r in range(0, case["N"], step):
                rows = slice(r, r + step)
                pairs = _pairs(case, s["keep"], b, h)[rows]
                z = (q[rows] @ k.T / math.sqrt(case["d"])).masked_fill(~pairs, -1e300)
                o = (torch.softmax(z, 1) * pairs.any(1, keepdim=True)) @ v
                got = torch.autograd.grad(o, (q, k, v), s["dout"][b, h, rows].double())
                grads[0][b, h, rows] = got[0][rows]
                total = [t + g for t, g in zip(total, got[1:])]
            grads[1][b, h], grads[2][b, h] = total
    return tuple(grads)
