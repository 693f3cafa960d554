"""What is measured of the operators next to the sparse attention path: rotary
positions, layer norm with its gradient, the append to the key caches and the
dense attention over the latent cache.

`run` computes a case either in plain torch operations (own = False) or by the
package's calls (own = True); `exact` gives the same outputs from the
definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BASE = 10000.0
YARN = {"factor": 16.0, "orig_context": 4096, "beta_fast": 32.0, "beta_slow": 1.0}
EPS = 1e-6
QK, DV, IDX = 576, 512, 128     # latent row, its value part, indexer key


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step: the RoPE part of 64 sequences' queries, written
        # into the last 64 dims of the 576-dim attention queries
        {"name": "rope decode q", "op": "rope", "batch": 64, "tokens": 1, "heads": 128, "dim": 64,
         "rot": 64, "begin": 0, "half": False, "yarn": True, "type": "bf16", "back": False,
         "pos": 32000, "into": 576},
        # prefill of the indexer queries: 64 of each head's 128 dims turn
        {"name": "rope prefill index q", "op": "rope", "batch": 1, "tokens": 16384, "heads": 64,
         "dim": 128, "rot": 64, "begin": 0, "half": True, "yarn": True, "type": "bf16",
         "back": False, "pos": 0, "into": 0},
        # the warm-up loss's gradient of the indexer queries, carried back
        {"name": "rope gradient index q", "op": "rope", "batch": 1, "tokens": 4096, "heads": 64,
         "dim": 128, "rot": 64, "begin": 0, "half": True, "yarn": False, "type": "f32",
         "back": True, "pos": 0, "into": 0},
        # the indexer keys of one decode step
        {"name": "norm decode keys", "op": "norm", "rows": 64, "dim": 128, "type": "bf16"},
        # the indexer keys of a 64K prefill
        {"name": "norm prefill keys", "op": "norm", "rows": 65536, "dim": 128, "type": "bf16"},
        # their gradient: fp32 from the warm-up loss, bf16 to the projection
        {"name": "norm gradient keys", "op": "norm_back", "rows": 65536, "dim": 128,
         "type": "bf16", "grad": "f32"},
        # wide rows of a residual stream, a ragged number of them, in training
        {"name": "norm gradient wide", "op": "norm_back", "rows": 8191, "dim": 4096,
         "type": "f32", "grad": "f32"},
        # one decode step's tokens into the paged caches
        {"name": "append decode", "op": "append", "batch": 64, "tokens": 1, "room": 1024,
         "page": 128, "pos": 700},
        # ragged prompts in a padded batch
        {"name": "append prefill", "op": "append", "batch": 8, "tokens": 4099, "room": 8192,
         "page": 256, "pos": 1000},
        # few sequences with short, ragged contexts, four tokens at once
        {"name": "dense short", "op": "dense", "batch": 8, "tokens": 4, "heads": 128, "low": 1,
         "high": 1500, "page": 128},
        # one long sequence: the cache is all there is to split
        {"name": "dense one long", "op": "dense", "batch": 1, "tokens": 1, "heads": 128,
         "low": 65536, "high": 65536, "page": 0},
        # a full decode batch over ragged long contexts, paged
        {"name": "dense batch", "op": "dense", "batch": 64, "tokens": 1, "heads": 128,
         "low": 16384, "high": 32768, "page": 256},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rope", "norm", "norm_back", "append", "dense", "dense"])
    if op == "rope":
        rot = 2 * _spread(rng, 4, 64)
        begin = rng.choice([0, 0, 8, 3])
        dim = begin + rot + rng.choice([0, 0, 16, 64, 5])
        heads = _spread(rng, 1, 128)
        most = max(2, 130_000_000 // (heads * dim))
        batch = _spread(rng, 1, min(64, most))
        return {"op": op, "batch": batch, "tokens": _spread(rng, 1, max(1, min(16384, most // batch))),
                "heads": heads, "dim": dim, "rot": rot, "begin": begin,
                "half": rng.random() < 0.5, "yarn": rng.random() < 0.5,
                "type": rng.choice(["bf16", "f32"]), "back": rng.random() < 0.4,
                "pos": _spread(rng, 1, 200_000), "into": rng.choice([0, 0, dim + 64, dim + 7])}
    if op in ("norm", "norm_back"):
        dim = rng.choice([128, 128, _spread(rng, 1, 8192), 8 * _spread(rng, 4, 1024)])
        case = {"op": op, "rows": _spread(rng, 1, max(2, min(65536, 33_000_000 // dim))),
                "dim": dim, "type": rng.choice(["bf16", "f32"])}
        if op == "norm_back":
            case["grad"] = rng.choice(["bf16", "f32"])
        return case
    if op == "append":
        page = rng.choice([0, 128, 256, 1024])
        room = _spread(rng, 128, 8192)
        tokens = _spread(rng, 1, min(room, 4096))
        return {"op": op, "batch": _spread(rng, 1, max(1, min(64, 65536 // room))),
                "tokens": tokens, "room": room, "page": page,
                "pos": rng.randrange(0, room - tokens + 1)}
    high, tokens = _spread(rng, 1, 65536), rng.choice([1, 1, 1, 2, 4])
    return {"op": op, "batch": _spread(rng, 1, max(1, min(64, 1_000_000 // (high * tokens)))),
            "tokens": tokens, "heads": rng.choice([128, 128, 64, 16, 33]),
            "low": max(1, high // rng.choice([1, 2, 8])), "high": high,
            "page": rng.choice([0, 128, 256, 1024])}


# ------------------------------------------------------------------ inputs

def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _spans(case):
    """Lengths between the case's low and high, one per sequence."""
    low, high, n = case["low"], case["high"], case["batch"]
    return [high if i == 0 else low + int((high - low) * ((i * 0.6180339887) % 1.0)) for i in range(n)]


def _fills(case):
    """New tokens per sequence of an append: the first sequence's are all there."""
    n = case["tokens"]
    return [n if i == 0 else max(1, n - int(n * 0.5 * ((i * 0.6180339887) % 1.0)))
            for i in range(case["batch"])]


def _table(g, batch, room, page):
    """A block table over a pool in random page order, and the pool's rows."""
    if not page:
        return None, batch * room
    per = -(-room // page)
    pages = torch.randperm(batch * per, generator=g, device=DEV).to(torch.int32)
    return pages.view(batch, per).contiguous(), batch * per * page


def _rows(table, page, batch, room):
    """Cache row of every (sequence, position)."""
    s = torch.arange(room, device=DEV)
    if table is None:
        return torch.arange(batch, device=DEV)[:, None] * room + s
    return table.long()[:, s // page] * page + s % page


def _frequencies(rot, yarn):
    """Radians per position of each pair; YaRN's blend of scaled and plain ones."""
    out = []
    for i in range(rot // 2):
        f = BASE ** (-2.0 * i / rot)
        if yarn:
            turns = YARN["orig_context"] * f / (2 * math.pi)
            keep = (turns - YARN["beta_slow"]) / (YARN["beta_fast"] - YARN["beta_slow"])
            keep = min(1.0, max(0.0, keep))
            f = (1 - keep) * f / YARN["factor"] + keep * f
        out.append(f)
    return out


def _amplitude(yarn):
    return 0.1 * math.log(YARN["factor"]) + 1.0 if yarn else 1.0


def _spec(dsa, rot, begin, half, yarn):
    return dsa.rope_spec(rot, rot_begin=begin, base=BASE,
                         layout=dsa.DSA_ROPE_HALF if half else dsa.DSA_ROPE_INTERLEAVED,
                         scaling=dsa.DSA_ROPE_YARN if yarn else dsa.DSA_ROPE_PLAIN,
                         amplitude=_amplitude(yarn), **(YARN if yarn else {}))


def prepare(case, seed):
    return {"rope": _prepare_rope, "norm": _prepare_norm, "norm_back": _prepare_norm_back,
            "append": _prepare_append, "dense": _prepare_dense}[case["op"]](case, _rng(seed))


def _prepare_rope(c, g):
    t = _type(c["type"])
    st = {"case": c, "x": _randn(g, c["batch"], c["tokens"], c["heads"], c["dim"], dtype=t),
          "freq": torch.tensor(_frequencies(c["rot"], c["yarn"]), dtype=torch.float64, device=DEV)}
    pos0 = [c["pos"] + 17 * b for b in range(c["batch"])]
    st["pos0"] = torch.tensor(pos0, dtype=torch.int32, device=DEV)
    wide = torch.zeros(c["batch"], c["tokens"], c["heads"], c["into"] or c["dim"], dtype=t, device=DEV)
    st["out"] = wide[..., wide.shape[-1] - c["dim"]:]
    if own:
        import sparse_attention_long_fp8_b200 as dsa
        st["spec"] = _spec(dsa, c["rot"], c["begin"], c["half"], c["yarn"])
    return st


def _prepare_norm(c, g):
    t = _type(c["type"])
    n, d = c["rows"], c["dim"]
    return {"case": c, "x": (_randn(g, n, d) * 2 + 0.5).to(t), "w": 1 + 0.2 * _randn(g, d),
            "b": 0.1 * _randn(g, d), "y": torch.empty(n, d, dtype=t, device=DEV),
            "mean": torch.empty(n, device=DEV), "rstd": torch.empty(n, device=DEV)}


def _prepare_norm_back(c, g):
    st = _prepare_norm(c, g)
    st["dy"] = _randn(g, c["rows"], c["dim"]).to(_type(c["grad"]))
    x = st["x"].float()
    st["mean"] = x.mean(-1)
    st["rstd"] = (x - st["mean"][:, None]).square().mean(-1).add(EPS).rsqrt()
    st["dx"], st["dw"], st["db"] = torch.empty_like(st["x"]), torch.empty_like(st["w"]), torch.empty_like(st["b"])
    if own:
        import sparse_attention_long_fp8_b200 as dsa
        st["ws_bytes"] = dsa.layernorm_bwd_workspace(c["rows"], c["dim"])
        st["ws"] = torch.empty(max(256, st["ws_bytes"]), dtype=torch.uint8, device=DEV)
    return st


def _prepare_append(c, g):
    B, n, room = c["batch"], c["tokens"], c["room"]
    table, pool = _table(g, B, room, c["page"])
    st = {"case": c, "table": table,
          "k": (_randn(g, B, n, IDX) * 2 + 0.5).bfloat16(), "c": _randn(g, B, n, QK, dtype=torch.bfloat16),
          "w": 1 + 0.2 * _randn(g, IDX), "b": 0.1 * _randn(g, IDX),
          "freq": torch.tensor(_frequencies(64, True), dtype=torch.float64, device=DEV),
          "pos0": torch.tensor([c["pos"] if i == 0 else int(c["pos"] * ((i * 0.7548776662) % 1.0))
                                for i in range(B)], dtype=torch.int32, device=DEV),
          "new": torch.tensor(_fills(c), dtype=torch.int32, device=DEV),
          "codes": torch.zeros(pool, IDX, dtype=torch.uint8, device=DEV),
          "scale": torch.ones(pool, device=DEV),
          "kv": torch.zeros(pool, QK, dtype=torch.bfloat16, device=DEV)}
    if own:
        import sparse_attention_long_fp8_b200 as dsa
        st["shape"] = dsa.DsaShape(B, n, room, 64, IDX, 2048, 128, QK, DV, 1.0 / 24.0)
        st["layout"] = None if table is None else dsa.make_layout(None, table, c["page"], pool)
        st["spec_k"] = _spec(dsa, 64, 0, True, True)
        st["spec_c"] = _spec(dsa, 64, 512, False, True)
    return st


def _prepare_dense(c, g):
    B, n, room = c["batch"], c["tokens"], c["high"]
    table, pool = _table(g, B, room, c["page"])
    kv = _randn(g, pool, QK, dtype=torch.bfloat16)
    hot = torch.rand(pool, 1, generator=g, device=DEV) < 0.05
    u = _randn(g, QK)
    kv += torch.where(hot, (3.0 * u * (math.sqrt(QK) / u.norm())).bfloat16(), torch.zeros((), dtype=torch.bfloat16, device=DEV))
    lens = torch.tensor(_spans(c), dtype=torch.int32, device=DEV)
    st = {"case": c, "table": table, "kv": kv, "lens": lens, "pos0": lens - n,
          "q": _randn(g, B, n, c["heads"], QK, dtype=torch.bfloat16),
          "out": torch.empty(B, n, c["heads"], DV, dtype=torch.bfloat16, device=DEV),
          "lse": torch.empty(B, n, c["heads"], device=DEV)}
    if own:
        import sparse_attention_long_fp8_b200 as dsa
        st["shape"] = dsa.DsaShape(B, n, room, 64, IDX, 2048, c["heads"], QK, DV, 1.0 / 24.0)
        st["layout"] = None if table is None else dsa.make_layout(None, table, c["page"], pool)
        st["ws"], st["ws_bytes"] = dsa.alloc_workspace(st["shape"], dsa.DSA_OP_DENSE_ATTN)
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "norm": _own_norm, "norm_back": _own_norm_back,
                "append": _own_append, "dense": _own_dense}[op](state)
    return {"rope": _plain_rope, "norm": _plain_norm, "norm_back": _plain_norm_back,
            "append": _plain_append, "dense": _plain_dense}[op](state)


def _own_rope(st):
    import sparse_attention_long_fp8_b200 as dsa
    dsa.dsa_rope(st["spec"], st["x"], st["out"], q_pos0=st["pos0"], backward=st["case"]["back"])
    return st["out"]


def _own_norm(st):
    import sparse_attention_long_fp8_b200 as dsa
    dsa.dsa_layernorm(st["x"], st["w"], st["b"], EPS, st["y"], st["mean"], st["rstd"])
    return {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}


def _own_norm_back(st):
    import sparse_attention_long_fp8_b200 as dsa
    dsa.dsa_layernorm_bwd(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], st["dx"], st["dw"],
                          st["db"], st["ws"], st["ws_bytes"])
    return {"dx": st["dx"], "dw": st["dw"], "db": st["db"]}


def _own_append(st):
    import sparse_attention_long_fp8_b200 as dsa
    dsa.dsa_cache_append(st["shape"], st["k"], st["w"], st["b"], EPS, st["spec_k"], st["c"],
                         st["spec_c"], st["pos0"], st["new"], st["codes"], st["scale"], st["kv"],
                         layout=st["layout"])
    return {"codes": st["codes"].view(torch.float8_e4m3fn), "scale": st["scale"], "kv": st["kv"]}


def _own_dense(st):
    import sparse_attention_long_fp8_b200 as dsa
    dsa.dsa_dense_attn(st["shape"], st["q"], st["kv"], st["pos0"], st["lens"], st["out"], st["lse"],
                       st["ws"], st["ws_bytes"], layout=st["layout"])
    return {"out": st["out"], "lse": st["lse"]}


def _turn(x, pos, freq, begin, half, amplitude, back):
    """x [B, T, H, D] in 32 bits, turned by its positions [B, T]; the angles in 64."""
    rot = 2 * freq.numel()
    angle = pos.double()[:, :, None, None] * freq
    cos, sin = (angle.cos() * amplitude).float(), (angle.sin() * amplitude).float()
    if back:
        sin = -sin
    part = x[..., begin:begin + rot]
    if half:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([x[..., :begin], turned, x[..., begin + rot:]], -1)


def _plain_rope(st):
    c = st["case"]
    pos = st["pos0"][:, None] + torch.arange(c["tokens"], device=DEV)
    y = _turn(st["x"].float(), pos, st["freq"], c["begin"], c["half"], _amplitude(c["yarn"]), c["back"])
    return y.to(st["x"].dtype)


def _norm_stats(x):
    mean = x.mean(-1)
    return mean, ((x - mean[..., None]).square().mean(-1) + EPS).rsqrt()


def _plain_norm(st):
    x = st["x"].float()
    mean, rstd = _norm_stats(x)
    y = (x - mean[:, None]) * rstd[:, None] * st["w"] + st["b"]
    return {"y": y.to(st["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_back(st):
    x, dy, rstd = st["x"].float(), st["dy"].float(), st["rstd"][:, None]
    hat = (x - st["mean"][:, None]) * rstd
    g = dy * st["w"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - hat * (g * hat).mean(-1, keepdim=True))
    return {"dx": dx.to(st["x"].dtype), "dw": (dy * hat).sum(0), "db": dy.sum(0)}


def _plain_append(st):
    c = st["case"]
    B, n = c["batch"], c["tokens"]
    i = torch.arange(n, device=DEV)
    pos = st["pos0"].long()[:, None] + i
    there = i < st["new"][:, None]
    rows = _rows(st["table"], c["page"], B, c["room"]).gather(1, pos.clamp(max=c["room"] - 1))[there]
    k = st["k"].float()
    mean, rstd = _norm_stats(k)
    k = (k - mean[..., None]) * rstd[..., None] * st["w"] + st["b"]
    k = _turn(k[:, :, None], pos, st["freq"], 0, True, _amplitude(True), False)[:, :, 0]
    amax = k.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (k / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    kv = _turn(st["c"].float()[:, :, None], pos, st["freq"], 512, False, _amplitude(True), False)[:, :, 0]
    st["codes"][rows] = codes[there]
    st["scale"][rows] = scale[there]
    st["kv"][rows] = kv[there].bfloat16()
    return {"codes": st["codes"].view(torch.float8_e4m3fn), "scale": st["scale"], "kv": st["kv"]}


def _plain_dense(st):
    c = st["case"]
    B, n, H, room = c["batch"], c["tokens"], c["heads"], c["high"]
    kv = st["kv"][_rows(st["table"], c["page"], B, room)].float()
    s = torch.bmm(st["q"].float().view(B, n * H, QK), kv.transpose(1, 2)) * (1.0 / 24.0)
    pos = st["pos0"][:, None] + torch.arange(n, device=DEV)
    last = torch.minimum(pos + 1, st["lens"][:, None])
    seen = torch.arange(room, device=DEV) < last[:, :, None]
    s = s.view(B, n, H, room).masked_fill_(~seen[:, :, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p.view(B, n * H, room), kv[..., :DV]).view(B, n, H, DV)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return {"out": out.bfloat16(), "lse": (top + total.log())[..., 0]}


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "rope":
        n = c["batch"] * c["tokens"] * c["heads"]
        size = 2 if c["type"] == "bf16" else 4
        return {"bytes": 2 * n * c["dim"] * size + 4 * c["batch"], "flops": 3 * n * c["rot"]}
    if c["op"] == "norm":
        n, d, size = c["rows"], c["dim"], 2 if c["type"] == "bf16" else 4
        return {"bytes": 2 * n * d * size + 8 * d + 8 * n, "flops": 8 * n * d}
    if c["op"] == "norm_back":
        n, d, size = c["rows"], c["dim"], 2 if c["type"] == "bf16" else 4
        grad = 2 if c["grad"] == "bf16" else 4
        return {"bytes": n * d * (2 * size + grad) + 8 * n + 12 * d, "flops": 14 * n * d}
    if c["op"] == "append":
        n = sum(_fills(c))
        return {"bytes": n * (2 * (IDX + QK) + IDX + 4 + 2 * QK) + 8 * IDX + 8 * c["batch"],
                "flops": n * (12 * IDX + 6 * 64)}
    spans, n, H = _spans(c), c["tokens"], c["heads"]
    pairs = sum(max(0, s - n + 1 + i) for s in spans for i in range(n))
    rows = c["batch"] * n * H
    return {"bytes": 2 * QK * sum(spans) + rows * (2 * QK + 2 * DV + 4) + 8 * c["batch"],
            "flops": 2 * H * (QK + DV) * pairs}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "norm": _exact_norm, "norm_back": _exact_norm_back,
            "append": _exact_append, "dense": _exact_dense}[case["op"]](st)


def _exact_turn(x, pos, c):
    """x [..., D] in 64 bits with pos [...]: pairs as complex numbers times e^(i pos f)."""
    y = x.clone()
    half = c["rot"] // 2
    for i, f in enumerate(_frequencies(c["rot"], c["yarn"])):
        a, b = (i, i + half) if c["half"] else (2 * i, 2 * i + 1)
        angle = pos.double() * (-f if c["back"] else f)
        z = torch.complex(x[..., c["begin"] + a], x[..., c["begin"] + b])
        z = z * torch.polar(torch.full_like(angle, _amplitude(c["yarn"])), angle)
        y[..., c["begin"] + a], y[..., c["begin"] + b] = z.real, z.imag
    return y


def _exact_rope(st):
    c = st["case"]
    pos = (st["pos0"].double()[:, None] + torch.arange(c["tokens"], device=DEV))[:, :, None]
    return _exact_turn(st["x"].double(), pos.expand(-1, -1, c["heads"]), c)


def _exact_hat(x):
    mean = x.mean(-1, keepdim=True)
    rstd = 1.0 / ((x * x).mean(-1, keepdim=True) - mean * mean + EPS).sqrt()
    return mean, rstd, (x - mean) * rstd


def _exact_norm(st):
    mean, rstd, hat = _exact_hat(st["x"].double())
    return {"y": torch.addcmul(st["b"].double(), hat, st["w"].double()), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _exact_norm_back(st):
    x, dy = st["x"].double(), st["dy"].double()
    hat = (x - st["mean"].double()[:, None]) * st["rstd"].double()[:, None]
    d, g = x.shape[-1], dy * st["w"].double()
    dots = torch.einsum("nd,nd->n", g, hat)[:, None]
    dx = (g - (g.sum(-1, keepdim=True) + hat * dots) / d) * st["rstd"].double()[:, None]
    ones = torch.ones(x.shape[0], dtype=torch.float64, device=DEV)
    return {"dx": dx, "dw": ones @ (dy * hat), "db": ones @ dy}


def _exact_append(st):
    c = st["case"]
    codes = torch.zeros(st["codes"].shape, dtype=torch.float64, device=DEV)
    scale, kv = st["scale"].double(), st["kv"].double()
    turn = {"rot": 64, "begin": 0, "half": True, "yarn": True, "back": False}
    rows = _rows(st["table"], c["page"], c["batch"], c["room"])
    for b, n in enumerate(_fills(c)):
        pos = int(st["pos0"][b]) + torch.arange(n, device=DEV)
        at = rows[b, pos]
        k = _exact_hat(st["k"][b, :n].double())[2] * st["w"].double() + st["b"].double()
        k = _exact_turn(k, pos, turn)
        amax = k.abs().amax(-1)
        step = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        codes[at] = (k / step[:, None]).float().to(torch.float8_e4m3fn).double()
        scale[at] = step
        kv[at] = _exact_turn(st["c"][b, :n].double(), pos, {**turn, "begin": 512, "half": False})
    return {"codes": codes, "scale": scale, "kv": kv}


def _exact_dense(st):
    c = st["case"]
    rows = _rows(st["table"], c["page"], c["batch"], c["high"])
    out, lse = st["out"].double(), st["lse"].double()
    for b, s in enumerate(_spans(c)):
        kv = st["kv"][rows[b, :s]].double()
        for i in range(c["tokens"]):
            n = min(s, s - c["tokens"] + i + 1)
            if n < 1:
                out[b, i], lse[b, i] = 0.0, float("-inf")
                continue
            logits = torch.einsum("hd,kd->hk", st["q"][b, i].double(), kv[:n]) / 24.0
            lse[b, i] = torch.logsumexp(logits, -1)
            out[b, i] = torch.softmax(logits, -1) @ kv[:n, :DV]
    return {"out": out, "lse": lse}
