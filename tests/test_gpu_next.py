"""GPU parity of the operators next to the sparse path against their formulas
in 64 bits: rotary positions, layer norm and its gradient, cache append, dense
attention, and runs of them together.

Tolerances count roundings: U = 2^-24 is half a step of fp32, HALF[t] that of
the output type. fp32 sums of n terms are off by at most (their longest chain
of additions) * U * sum of the terms' sizes.
"""
import math

import pytest
import torch

import sparse_attention_long_fp8_b200 as dsa

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean():
    dsa.dsa_check()
    yield
    torch.cuda.synchronize()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _within(got, want, tol, what):
    got, want = got.double(), want.double()
    err = (got - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float(err[bad].max()):.3e}"


# ------------------------------------------------------------------ rotary positions

def _turn64(x, pos, spec, back=False):
    """(turned, size bound of the pair) in 64 bits; x [B, T, H, D], pos [B, T]."""
    x = x.double()
    P = spec.rot_dim // 2
    f = torch.tensor(list(spec.freq[:P]), dtype=torch.float64, device=x.device)
    a = pos.double()[:, :, None, None] * f
    c, s = a.cos() * spec.amplitude, a.sin() * spec.amplitude * (-1 if back else 1)
    y, size = x.clone(), torch.zeros_like(x)
    b0 = spec.rot_begin
    if spec.layout == dsa.DSA_ROPE_HALF:
        i, j = slice(b0, b0 + P), slice(b0 + P, b0 + 2 * P)
    else:
        i, j = slice(b0, b0 + 2 * P, 2), slice(b0 + 1, b0 + 2 * P, 2)
    u, v = x[..., i], x[..., j]
    y[..., i], y[..., j] = u * c - v * s, u * s + v * c
    m = (u.abs() + v.abs()) * abs(spec.amplitude)
    size[..., i], size[..., j] = m, m
    return y, size


def _rope_tol(want, size, dtype):
    # angle: a float fraction of a turn, 2 pi 2^-26; sincospi 2 ulp = 2^-22;
    # amplitude, products and sum: 4 roundings. Together below 6e-7 of the pair.
    return size * 6e-7 + (want.abs() + size * 6e-7) * HALF[dtype]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [dsa.DSA_ROPE_HALF, dsa.DSA_ROPE_INTERLEAVED])
@pytest.mark.parametrize("B,T,H,D,rot,begin", [
    (1, 1, 1, 2, 2, 0), (1, 1, 128, 64, 64, 0), (2, 5, 3, 128, 64, 0), (3, 7, 1, 576, 64, 512),
    (1, 300, 5, 33, 10, 3), (2, 129, 2, 80, 48, 16), (1, 65, 1, 256, 256, 0), (4, 1, 7, 72, 40, 8),
    (2, 2500, 4, 128, 64, 32)])
def test_rope(B, T, H, D, rot, begin, layout, dtype):
    g = _gen(B * 1000 + T)
    x = _randn(g, B, T, H, D, dtype=dtype)
    pos0 = torch.randint(0, 70000, (B,), generator=g, device=DEV, dtype=torch.int32)
    pos = pos0[:, None] + torch.arange(T, device=DEV)
    spec = dsa.rope_spec(rot, rot_begin=begin, layout=layout, scaling=dsa.DSA_ROPE_YARN, factor=8.0,
                         orig_context=4096, amplitude=1.2)
    for back in (False, True):
        out = torch.full_like(x, 7.0)
        dsa.dsa_rope(spec, x, out, q_pos0=pos0, backward=back)
        want, size = _turn64(x, pos, spec, back)
        _within(out, want, _rope_tol(want, size, dtype), "rope")
        fixed = torch.ones(D, dtype=torch.bool, device=DEV)
        fixed[begin:begin + rot] = False
        assert torch.equal(out[..., fixed], x[..., fixed])
        y = x.clone()
        dsa.dsa_rope(spec, y, y, q_pos0=pos0, backward=back)      # in place
        assert torch.equal(y, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [dsa.DSA_ROPE_HALF, dsa.DSA_ROPE_INTERLEAVED])
@pytest.mark.parametrize("B,T,H,D,rot,begin,width,lead", [
    (2, 33, 3, 36, 20, 8, 36, 0), (1, 700, 2, 38, 28, 6, 44, 2), (3, 129, 5, 60, 44, 4, 124, 4),
    (2, 257, 64, 40, 24, 12, 48, 4), (1, 1500, 1, 31, 26, 0, 95, 1), (2, 40, 97, 150, 126, 8, 151, 0),
    (64, 3, 1, 8, 8, 0, 10, 2), (1, 5000, 3, 9, 2, 3, 9, 0)])
def test_rope_at_every_alignment(B, T, H, D, rot, begin, width, lead, layout, dtype):
    g = _gen(T + D)
    x = _randn(g, B, T, H, D, dtype=dtype)
    wide = torch.full((B, T, H, width), 7.0, device=DEV, dtype=dtype)
    out = wide[..., lead:lead + D]
    pos = torch.randint(0, 9000, (B, T), generator=g, device=DEV, dtype=torch.int32)
    pad = torch.rand(B, T, generator=g, device=DEV) < 0.1
    spec = dsa.rope_spec(rot, rot_begin=begin, layout=layout)
    dsa.dsa_rope(spec, x, out, row_pos=torch.where(pad, -1, pos).to(torch.int32))
    want, size = _turn64(x, pos, spec, False)
    want[pad], size[pad] = 7.0, 0.0
    _within(out, want, _rope_tol(want, size, dtype), "rope")
    assert (wide[..., :lead] == 7.0).all() and (wide[..., lead + D:] == 7.0).all()
    y = torch.full_like(wide, 3.0)[..., lead:lead + D]
    y.copy_(x)
    dsa.dsa_rope(spec, y, y, row_pos=torch.where(pad, -1, pos).to(torch.int32))    # in place
    assert torch.equal(y[~pad], out[~pad]) and torch.equal(y[pad], x[pad])


@pytest.mark.parametrize("pos", [0, 1, 1 << 20, (1 << 31) - 2])
def test_rope_far_positions(pos):
    g = _gen(3)
    x = _randn(g, 1, 1, 4, 64)
    p = torch.tensor([[pos]], dtype=torch.int32, device=DEV)
    spec = dsa.rope_spec(64)
    out = torch.empty_like(x)
    dsa.dsa_rope(spec, x, out, row_pos=p)
    want, size = _turn64(x, p, spec)
    # the reference's own product pos * f carries 2^-53 of up to 2^31 radians
    _within(out, want, _rope_tol(want, size, torch.float32) + size * 2.0 ** -21 * (pos > 1 << 20), "rope")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_strides_and_padding(dtype):
    g = _gen(5)
    B, T, H = 3, 6, 8
    wide = _randn(g, B, T, H, 200, dtype=dtype)
    spec = dsa.rope_spec(64, layout=dsa.DSA_ROPE_INTERLEAVED)
    pos = torch.randint(0, 1000, (B, T), generator=g, device=DEV, dtype=torch.int32)
    pos[1, 3:] = -1
    pos[2, 0] = -5
    for off in (128, 130):                                        # 16-byte aligned or not
        q = torch.full((B, T, H, 576), 3.0, device=DEV, dtype=dtype)
        x, out = wide[..., off:off + 64], q[..., 512:]
        dsa.dsa_rope(spec, x, out, row_pos=pos)
        want, size = _turn64(x, pos, spec)
        there = pos >= 0
        _within(out[there], want[there], _rope_tol(want, size, dtype)[there], "rope")
        assert (out[~there] == 3.0).all() and (q[..., :512] == 3.0).all()
    # heads ahead of tokens, and a head that all share
    y = _randn(g, B, H, T, 64, dtype=dtype).transpose(1, 2)
    z = _randn(g, B, T, 1, 64, dtype=dtype).expand(B, T, H, 64)
    pos = pos.clamp_min(0)
    for x in (y, z):
        out = torch.empty(B, H, T, 64, device=DEV, dtype=dtype).transpose(1, 2)
        dsa.dsa_rope(spec, x, out, row_pos=pos)
        want, size = _turn64(x, pos, spec)
        _within(out, want, _rope_tol(want, size, dtype), "rope")
    # one slice of a buffer into another of the same rows
    a = wide.clone()
    dsa.dsa_rope(spec, a[..., :64], a[..., 64:128], row_pos=pos)
    want, size = _turn64(wide[..., :64], pos, spec)
    _within(a[..., 64:128], want, _rope_tol(want, size, dtype), "rope")
    assert torch.equal(a[..., :64], wide[..., :64]) and torch.equal(a[..., 128:], wide[..., 128:])
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rope(spec, a[..., :64], a[..., 32:96], row_pos=pos)


def test_rope_gradient_against_differences():
    g = _gen(6)
    spec = dsa.rope_spec(32, rot_begin=8, amplitude=0.9)
    x, dy = _randn(g, 1, 3, 2, 48), _randn(g, 1, 3, 2, 48)
    dx, up, down = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dsa.dsa_rope(spec, dy, dx, backward=True)
    d = _randn(g, 1, 3, 2, 48)
    dsa.dsa_rope(spec, x + d, up)
    dsa.dsa_rope(spec, x - d, down)
    # linear, so the central difference is exact up to rounding: 48 * 6 terms
    # of size < 30, each off by 1e-6 of it
    lhs = ((up - down).double() * dy.double()).sum() / 2
    assert abs(float(lhs - (dx.double() * d.double()).sum())) < 288 * 30 * 1e-6


# ------------------------------------------------------------------ layer norm

NORMS = [(1, 1), (3, 7), (5, 8), (64, 128), (1000, 128), (17, 129), (33, 256), (9, 500), (700, 512),
         (5, 1000), (6, 1024), (4, 2040), (3, 4096), (300, 2056), (3, 4097), (2, 8192), (2, 16384), (2, 16381)]


def _norm64(x, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    return mean, rstd, (x - mean) * rstd


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", NORMS)
def test_layernorm(rows, dim, dtype):
    g = _gen(rows + dim)
    x = (_randn(g, rows, dim) * 2 + 30.0).to(dtype)
    w, b = _randn(g, dim), _randn(g, dim)
    for weight, bias in ((w, b), (None, None)):
        y, mean, rstd = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        dsa.dsa_layernorm(x, weight, bias, 1e-5, y, mean, rstd)
        m, r, hat = _norm64(x, 1e-5)
        ww = (weight if weight is not None else torch.ones_like(w)).double()
        bb = (bias if bias is not None else torch.zeros_like(b)).double()
        want = hat * ww + bb
        # sums: at most 16 in a thread, 5 + 32 across threads, divisions: 64
        size = x.double().abs().mean(-1, keepdim=True)
        _within(mean[:, None], m, size * 64 * U, "mean")
        # d var = 2 (x - mean) d mean sums to 0 up to second order; its terms 64 roundings
        lost = (size * 64 * U) ** 2 * r * r
        _within(rstd[:, None], r, r * (64 * U + lost), "rstd")
        tol = ww.abs() * (hat.abs() * (70 * U + lost) + r * size * 64 * U) + (want.abs() + bb.abs()) * 4 * U
        _within(y, want, tol + (want.abs() + tol) * HALF[dtype], "y")


@pytest.mark.parametrize("xt,gt,dt", [(torch.bfloat16, torch.float32, torch.bfloat16),
                                      (torch.float32, torch.float32, torch.float32),
                                      (torch.bfloat16, torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("rows,dim", NORMS)
def test_layernorm_gradient(rows, dim, xt, gt, dt):
    g = _gen(rows * 3 + dim)
    x, dy, w = (_randn(g, rows, dim) * 2 - 1).to(xt), _randn(g, rows, dim, dtype=gt), _randn(g, dim)
    m, r, _ = _norm64(x, 1e-6)
    mean, rstd = m[:, 0].float(), r[:, 0].float()
    n = dsa.layernorm_bwd_workspace(rows, dim)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    hat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for weight in (w, None):
        dx = torch.empty(rows, dim, device=DEV, dtype=dt)
        dw, db = torch.full((dim,), 9.0, device=DEV), torch.full((dim,), 9.0, device=DEV)
        dsa.dsa_layernorm_bwd(dy, x, weight, mean, rstd, dx, dw, db, ws, n)
        d = dy.double()
        q = d * (weight.double() if weight is not None else 1.0)
        want = rstd.double()[:, None] * (q - q.mean(-1, keepdim=True) - hat * (q * hat).mean(-1, keepdim=True))
        size = rstd.double()[:, None] * (q.abs() + q.abs().mean(-1, keepdim=True)
                                         + hat.abs() * (q * hat).abs().mean(-1, keepdim=True))
        _within(dx, want, size * 72 * U + (want.abs() + size * 72 * U) * HALF[dt], "dx")
        # columns: at most 8 rows in a thread here, 8 + 32 + 5 sums after that
        _within(dw, (d * hat).sum(0), (d * hat).abs().sum(0) * 64 * U, "dweight")
        _within(db, d.sum(0), d.abs().sum(0) * 64 * U, "dbias")
    # the same bits again; without the sums, the same dx
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    dsa.dsa_layernorm_bwd(dy, x, None, mean, rstd, dx2, dw2, db2, ws, n)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    dsa.dsa_layernorm_bwd(dy, x, None, mean, rstd, dx2.zero_())
    assert torch.equal(dx, dx2)


def test_layernorm_gradient_against_differences():
    g = _gen(8)
    rows, dim = 5, 40
    x, w, b, dy = _randn(g, rows, dim), _randn(g, dim), _randn(g, dim), _randn(g, rows, dim)
    mean, rstd, y = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty_like(x)
    dsa.dsa_layernorm(x, w, b, 1e-6, y, mean, rstd)
    n = dsa.layernorm_bwd_workspace(rows, dim)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    dsa.dsa_layernorm_bwd(dy, x, w, mean, rstd, dx, dw, db, ws, n)

    def loss(x, w, b):
        _, _, hat = _norm64(x, 1e-6)
        return ((hat * w.double() + b.double()) * dy.double()).sum()
    for t, grad in (("x", dx), ("w", dw), ("b", db)):
        v = {"x": x, "w": w, "b": b}
        d = _randn(g, *v[t].shape).double()
        h = 1e-4
        hi = loss(**{k: (u.double() + h * d if k == t else u.double()) for k, u in v.items()})
        lo = loss(**{k: (u.double() - h * d if k == t else u.double()) for k, u in v.items()})
        # third derivative times h^2 ~ 1e-8 of terms of size ~1; fp32 gradient 200 terms * 72 U
        assert abs(float((hi - lo) / (2 * h) - (grad.double() * d).sum())) < 1e-3, t


def test_layernorm_no_rows_strides_and_in_place():
    g = _gen(9)
    e = torch.empty(0, 128, device=DEV)
    dsa.dsa_layernorm(e, None, None, 1e-6, e)
    dw, db = torch.full((128,), 5.0, device=DEV), torch.full((128,), 5.0, device=DEV)
    z = torch.empty(0, device=DEV)
    dsa.dsa_layernorm_bwd(e, e, None, z, z, e, dw, db)
    assert (dw == 0).all() and (db == 0).all()
    wide = _randn(g, 50, 300, dtype=torch.bfloat16)
    out = torch.full((50, 200), 2.0, device=DEV)
    for lo in (8, 9):
        x, y = wide[:, lo:lo + 128], out[:, lo:lo + 128]
        mean, rstd = torch.empty(50, device=DEV), torch.empty(50, device=DEV)
        dsa.dsa_layernorm(x, None, None, 1e-6, y, mean, rstd)
        ref = torch.empty(50, 128, device=DEV)
        dsa.dsa_layernorm(x.contiguous(), None, None, 1e-6, ref)
        # aligned rows and others differ in the order of their sums
        tol = 64 * U * (ref.double().abs() + rstd.double()[:, None] * x.double().abs().mean(-1, keepdim=True)) * 2
        _within(y, ref, tol, "strided")
        assert (out[:, :lo] == 2.0).all() and (out[:, lo + 128:] == 2.0).all()
        out.fill_(2.0)
    x = _randn(g, 40, 128)
    y = torch.empty_like(x)
    dsa.dsa_layernorm(x, None, None, 1e-6, y)
    dsa.dsa_layernorm(x, None, None, 1e-6, x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("rows,dim", [(700, 128), (300, 512), (250, 2048), (600, 4096), (5, 16384), (40, 1001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layernorm_gradient_in_place(rows, dim, dtype):
    g = _gen(dim)
    x, dy, w = _randn(g, rows, dim, dtype=dtype), _randn(g, rows, dim, dtype=dtype), _randn(g, dim)
    mean, rstd, y = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty_like(x)
    dsa.dsa_layernorm(x, w, None, 1e-6, y, mean, rstd)
    z = x.clone()
    dsa.dsa_layernorm(z, w, None, 1e-6, z)
    assert torch.equal(z, y)
    want = torch.empty_like(x)
    dsa.dsa_layernorm_bwd(dy, x, w, mean, rstd, want)
    a, b = dy.clone(), x.clone()
    dsa.dsa_layernorm_bwd(a, x, w, mean, rstd, a)
    dsa.dsa_layernorm_bwd(dy, b, w, mean, rstd, b)
    assert torch.equal(a, want) and torch.equal(b, want)


@pytest.mark.parametrize("rows,dim", [(300, 128), (130, 1024), (600, 4096), (37, 72)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layernorm_between_columns_of_one_buffer(rows, dim, dtype):
    g = _gen(dim + rows)
    buf = _randn(g, rows, 3 * dim, dtype=dtype)
    x, dy, w = buf[:, dim:2 * dim], buf[:, :dim], _randn(g, dim)
    before = buf.clone()
    mean, rstd, want = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, dim, device=DEV,
                                                                                               dtype=dtype)
    dsa.dsa_layernorm(x, w, None, 1e-6, want, mean, rstd)
    dsa.dsa_layernorm(x, w, None, 1e-6, buf[:, 2 * dim:])
    assert torch.equal(buf[:, 2 * dim:], want) and torch.equal(buf[:, :2 * dim], before[:, :2 * dim])
    dsa.dsa_layernorm_bwd(dy, x, w, mean, rstd, want)
    dsa.dsa_layernorm_bwd(dy, x, w, mean, rstd, buf[:, 2 * dim:])
    assert torch.equal(buf[:, 2 * dim:], want) and torch.equal(buf[:, :2 * dim], before[:, :2 * dim])


# ------------------------------------------------------------------ cache append

def _cache(B, room, page, idx, qk, seed):
    """Empty caches with marked contents, contiguous or paged in random order."""
    g = _gen(seed)
    if page:
        per = -(-room // page)
        spare = 2
        perm = torch.randperm(B * per + spare, generator=g, device=DEV)[:B * per]
        table = perm.to(torch.int32).view(B, per).contiguous()
        pool = (B * per + spare) * page
        s = torch.arange(room, device=DEV)
        rows = table.long()[:, s // page] * page + s % page
        lay = dsa.make_layout(None, table, page, pool)
    else:
        table, pool, lay = None, B * room, None
        rows = torch.arange(B, device=DEV)[:, None] * room + torch.arange(room, device=DEV)
    return {"codes": torch.full((pool, idx), 0x55, dtype=torch.uint8, device=DEV),
            "scale": torch.full((pool,), 3.0, device=DEV),
            "kv": torch.full((pool, qk), 5.0, device=DEV, dtype=torch.bfloat16),
            "rows": rows, "layout": lay, "table": table}


@pytest.mark.parametrize("idx,qk", [(128, 576), (32, 64), (128, 64), (32, 576)])
@pytest.mark.parametrize("layout", [dsa.DSA_ROPE_HALF, dsa.DSA_ROPE_INTERLEAVED])
@pytest.mark.parametrize("B,T,room,page", [(1, 1, 1, 0), (5, 1, 300, 128), (3, 37, 200, 0), (4, 300, 513, 256)])
def test_append(B, T, room, page, layout, idx, qk):
    g = _gen(T * 7 + idx)
    k = (_randn(g, B, T, idx) * 3 + 1).bfloat16()
    c = _randn(g, B, T, qk, dtype=torch.bfloat16)
    w, b = _randn(g, idx), _randn(g, idx)
    new = torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    new[0] = T
    pos0 = (torch.rand(B, generator=g, device=DEV) * (room - T + 1)).to(torch.int32).clamp_max(room - T)
    ca = _cache(B, room, page, idx, qk, 11)
    was = {n: ca[n].clone() for n in ("codes", "scale", "kv")}
    rk = dsa.rope_spec(idx // 2, rot_begin=idx // 4, layout=layout, amplitude=1.1)
    rc = dsa.rope_spec(36, rot_begin=qk - 38, layout=layout)
    shape = dsa.DsaShape(B, T, room, 64, idx, 2048, 128, qk, 64, 1.0)
    dsa.dsa_cache_append(shape, k, w, b, 1e-6, rk, c, rc, pos0, new, ca["codes"], ca["scale"], ca["kv"],
                         layout=ca["layout"])
    dsa.dsa_check()
    i = torch.arange(T, device=DEV)
    pos = pos0[:, None] + i
    there = i < new[:, None]
    at = ca["rows"].gather(1, pos.long())[there]
    hit = torch.zeros(ca["scale"].numel(), dtype=torch.bool, device=DEV)
    hit[at] = True
    for n in was:
        assert torch.equal(ca[n][~hit], was[n][~hit]), n             # nothing else is touched
    want, size = _turn64(c[:, :, None], pos, rc)
    _within(ca["kv"][at], want[:, :, 0][there], _rope_tol(want, size, torch.bfloat16)[:, :, 0][there], "kv")
    # the key: sums of idx terms (40 roundings), norm and rotation 24 more
    _, r, hat = _norm64(k, 1e-6)
    key = hat * w.double() + b.double()
    slack = (hat.abs() + r * k.double().abs().mean(-1, keepdim=True)) * w.double().abs() + b.double().abs()
    want, _ = _turn64(key[:, :, None], pos, rk)
    _, slack_pair = _turn64(slack[:, :, None], pos, rk)
    want, slack = want[:, :, 0][there], torch.maximum(slack, slack_pair[:, :, 0])[there] * 64 * U
    amax = want.abs().amax(-1)
    _within(ca["scale"][at], amax / 448, slack.amax(-1) / 448 + amax / 448 * 2 * U, "scale")
    scale = ca["scale"][at].double()[:, None]
    got = ca["codes"][at].view(torch.float8_e4m3fn).double() * scale
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below 2^-6
    _within(got, want, torch.maximum(want.abs() * 2.0 ** -4, scale * 2.0 ** -10) + slack * 2, "codes")


def test_append_constant_key_and_reported_positions():
    # equal values normalise to the bias; with none the row is zero, scale 1
    shape = dsa.DsaShape(2, 2, 128, 64, 128, 2048, 128, 576, 512, 1.0)
    k = torch.full((2, 2, 128), 3.0, device=DEV, dtype=torch.bfloat16)
    c = torch.ones(2, 2, 576, device=DEV, dtype=torch.bfloat16)
    ca = _cache(2, 128, 128, 128, 576, 1)
    rk, rc = dsa.rope_spec(64), dsa.rope_spec(64, rot_begin=512)
    # positions past INT_MAX are reported, and nothing is written
    dsa.dsa_cache_append(shape, k, None, None, 1e-6, rk, c, rc,
                         torch.tensor([2147483647, -7], dtype=torch.int32, device=DEV), None, ca["codes"],
                         ca["scale"], ca["kv"], layout=ca["layout"])
    with pytest.raises(dsa.DsaError):
        dsa.dsa_check()
    assert (ca["scale"] == 3.0).all() and (ca["kv"] == 5.0).all()
    pos0 = torch.tensor([126, 127], dtype=torch.int32, device=DEV)   # the last token lies past the cache
    dsa.dsa_cache_append(shape, k, None, None, 1e-6, rk, c, rc, pos0, None, ca["codes"], ca["scale"],
                         ca["kv"], layout=ca["layout"])
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_check()
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG
    written = torch.cat([ca["rows"][0, 126:], ca["rows"][1, 127:]])
    assert (ca["scale"][written] == 1.0).all() and (ca["codes"][written] & 0x7f == 0).all()
    assert int((ca["scale"] != 3.0).sum()) == 3
    # pages outside the pool: nothing is written there or anywhere
    ca["table"][0, 0] = -1
    ca["table"][1, 0] = 4
    before = ca["kv"].clone()
    dsa.dsa_cache_append(shape, k, None, None, 1e-6, rk, c, rc, torch.zeros_like(pos0), None, ca["codes"],
                         ca["scale"], ca["kv"], layout=ca["layout"])
    with pytest.raises(dsa.DsaError):
        dsa.dsa_check()
    assert torch.equal(before, ca["kv"])


# ------------------------------------------------------------------ dense attention

def _dense_case(lens, T, H, page, seed, room=None, stale=float("nan")):
    """A latent cache whose rows past each length are `stale`."""
    g = _gen(seed)
    B = len(lens)
    room = room or max(max(lens), 1)
    ca = _cache(B, room, page, 128, 576, seed)
    ca["kv"].fill_(stale)
    for b, n in enumerate(lens):
        ca["kv"][ca["rows"][b, :n]] = _randn(g, n, 576, dtype=torch.bfloat16)
    q = _randn(g, B, T, H, 576, dtype=torch.bfloat16)
    kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return {"shape": dsa.DsaShape(B, T, room, 64, 128, 2048, H, 576, 512, 1.0 / 24), "q": q, "kv": ca["kv"],
            "kv_len": kv_len, "pos0": kv_len - T, "rows": ca["rows"], "layout": ca["layout"],
            "table": ca["table"]}


def _dense(c, dtype=torch.bfloat16, lse=True, ws=None, pos0="own", **kw):
    s = c["shape"]
    out = torch.full((s.batch, s.n_q, s.heads, 512), 9.0, device=DEV, dtype=dtype)
    l = torch.full((s.batch, s.n_q, s.heads), 9.0, device=DEV) if lse else None
    if ws is None:
        ws = dsa.alloc_workspace(s, dsa.DSA_OP_DENSE_ATTN)
    dsa.dsa_dense_attn(s, c["q"], c["kv"], c["pos0"] if isinstance(pos0, str) else pos0, c["kv_len"], out, l,
                       *ws, layout=kw.pop("layout", c["layout"]), **kw)
    return out, l


def _check_dense(c, out, lse, seen):
    """seen[b][i]: keys that the row sees."""
    s = c["shape"]
    for b in range(s.batch):
        for i in range(s.n_q):
            n = seen[b][i]
            if n <= 0:
                assert (out[b, i] == 0).all() and (lse[b, i] == -math.inf).all()
                continue
            kv = c["kv"][c["rows"][b, :n]].double()
            q = c["q"][b, i].double()
            logits = q @ kv.T * s.softmax_scale
            p = torch.softmax(logits, -1)
            want = p @ kv[:, :512]
            # logits: 576 products summed in fp32; p: that, ex2 (2^-22) and, for
            # O, half a bf16 step (2^-8), against the rows and their mean
            e = float((q.abs() @ kv.abs().T).max()) * s.softmax_scale * 600 * U
            tol = (2.0 ** -8 + 2 * e + 2.0 ** -20) * (p @ kv[:, :512].abs() + want.abs())
            _within(out[b, i], want, tol + (want.abs() + tol) * HALF[out.dtype], f"out {b} {i}")
            ref = torch.logsumexp(logits, -1)
            # one sum per block and warp, joined: n / 64 + 100 additions
            _within(lse[b, i], ref, e + (n / 64 + 100) * U + 2.0 ** -21 + ref.abs() * 4 * U, f"lse {b} {i}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,T,H,page", [
    ([1], 1, 128, 0), ([63], 1, 128, 0), ([64], 1, 1, 0), ([65], 1, 33, 0), ([129], 2, 128, 128),
    ([0, 5, 0, 200, 0], 1, 128, 128), ([0, 0], 1, 16, 0), ([1000], 4, 64, 256), ([7, 640, 128, 127], 3, 128, 0),
    ([9000], 1, 128, 1024), ([300] * 40, 2, 16, 128)])
def test_dense(lens, T, H, page, dtype):
    c = _dense_case(lens, T, H, page, sum(lens) + T)
    out, lse = _dense(c, dtype)
    dsa.dsa_check()
    _check_dense(c, out, lse, [[n - T + 1 + i for i in range(T)] for n in lens])
    again, _ = _dense(c, dtype, lse=False)
    assert torch.equal(out, again)                                   # the same bits, without lse too


@pytest.mark.parametrize("rows", [255, 257, 385, 1200])
def test_dense_many_rows(rows):
    # more rows than one warp, then than one block of threads holds at a time
    lens = [(i * 37) % 290 for i in range(rows)]
    c = _dense_case(lens, 1, 4, 128, rows)
    out, lse = _dense(c)
    dsa.dsa_check()
    _check_dense(c, out, lse, [[n] for n in lens])


@pytest.mark.parametrize("stale", [float("inf"), float("-inf"), 3e38])
def test_dense_never_uses_rows_past_the_length(stale):
    lens = [70, 1, 128, 383]
    a, b = _dense_case(lens, 1, 64, 128, 2, room=512, stale=0.0), _dense_case(lens, 1, 64, 128, 2, room=512, stale=stale)
    x, y = _dense(a), _dense(b)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_dense_positions_and_defaults():
    # no kv_len: the whole room; positions by row_pos, some before the cache
    c = _dense_case([200, 200], 3, 32, 0, 4)
    c["kv_len"] = None
    pos = torch.tensor([[0, 199, 63], [-1, 64, 2147483647]], dtype=torch.int32, device=DEV)
    out, lse = _dense(c, pos0=None, layout=dsa.make_layout(pos))
    _check_dense(c, out, lse, [[1, 200, 64], [0, 65, 200]])
    out, lse = _dense(c, pos0=None)                                  # positions 0, 1, 2
    _check_dense(c, out, lse, [[1, 2, 3]] * 2)
    # kv_len past the room counts as the room
    c["kv_len"] = torch.tensor([500, 100], dtype=torch.int32, device=DEV)
    out, lse = _dense(c, pos0=torch.tensor([400, 400], dtype=torch.int32, device=DEV))
    _check_dense(c, out, lse, [[200] * 3, [100] * 3])


def test_dense_visible_nan_and_infinity_come_through():
    c = _dense_case([130, 130], 1, 8, 0, 5)
    c["kv"][c["rows"][0, 129], 3] = math.nan
    out, lse = _dense(c)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert out[1].isfinite().all() and lse[1].isfinite().all()


def test_dense_large_logits_and_growing_maxima():
    # each block's keys outweigh the ones before: O is rescaled again and again
    c = _dense_case([640], 1, 128, 0, 6)
    ramp = torch.arange(640, device=DEV)[:, None] / 64.0
    c["kv"][:] = (c["kv"].float() * (1 + ramp)).bfloat16()
    out, lse = _dense(c, torch.float32)
    _check_dense(c, out, lse, [[640]])


def test_dense_page_outside_the_pool_counts_as_zeros():
    c = _dense_case([256, 100], 1, 16, 128, 7)
    zeroed = {**c, "kv": c["kv"].clone()}
    zeroed["kv"][c["rows"][0, 128:256]] = 0
    want = _dense(zeroed)
    dsa.dsa_check()
    for page in (-1, 1 << 20):
        c["table"][0, 1] = page
        got = _dense(c)
        with pytest.raises(dsa.DsaError) as e:
            dsa.dsa_check()
        assert e.value.status == dsa.DSA_ERR_INVALID_ARG
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_dense_equals_sparse_over_every_key():
    # the same keys named one by one to dsa_sparse_attn
    n = 1500
    c = _dense_case([n], 1, 128, 128, 8)
    s = c["shape"]
    s.topk = n
    idx = torch.arange(n, device=DEV, dtype=torch.int32).view(1, 1, n)
    out = torch.empty(1, 1, 128, 512, device=DEV)
    lse = torch.empty(1, 1, 128, device=DEV)
    ws = dsa.alloc_workspace(s, dsa.DSA_OP_SPARSE_ATTN)
    dsa.dsa_sparse_attn(s, c["q"], c["kv"], idx, out, lse, *ws, layout=c["layout"])
    d, l = _dense(c, torch.float32)
    _check_dense(c, d, l, [[n]])
    _check_dense(c, out, lse, [[n]])


def test_dense_graph_replays_with_other_lengths():
    c = _dense_case([900, 300], 1, 32, 128, 9)
    s = c["shape"]
    ws = dsa.alloc_workspace(s, dsa.DSA_OP_DENSE_ATTN)
    out, lse = torch.empty(2, 1, 32, 512, device=DEV, dtype=torch.bfloat16), torch.empty(2, 1, 32, device=DEV)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        dsa.dsa_dense_attn(s, c["q"], c["kv"], c["pos0"], c["kv_len"], out, lse, *ws, layout=c["layout"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            dsa.dsa_dense_attn(s, c["q"], c["kv"], c["pos0"], c["kv_len"], out, lse, *ws, layout=c["layout"])
        for lens in ([900, 300], [1, 299], [64, 0], [513, 65]):
            c["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
            c["pos0"].copy_(c["kv_len"] - 1)
            for _ in range(3):
                g.replay()
            st.synchronize()
            _check_dense(c, out, lse, [[n] for n in lens])
    torch.cuda.current_stream().wait_stream(st)


@pytest.mark.parametrize("lens", [[500], [513], [4000], [9473], [1000] * 4, [130, 0, 2500, 1], [1] * 7 + [3000]])
@pytest.mark.parametrize("T", [1, 2])
def test_dense_few_rows_in_shares_of_a_block(lens, T):
    c = _dense_case(lens, T, 33, 128, 40 + len(lens))
    out, lse = _dense(c)
    _check_dense(c, out, lse, [[n - T + 1 + i for i in range(T)] for n in lens])


def test_calls_at_once_on_two_streams():
    """Calls that overlap on the GPU, a workspace each: the results of the same
    calls one after another."""
    cases = [_dense_case([3000, 77, 1500], 1, 128, 128, 51), _dense_case([700] * 40, 2, 64, 256, 52)]
    g = _gen(53)
    x, dy, w = _randn(g, 5000, 128, dtype=torch.bfloat16), _randn(g, 5000, 128, dtype=torch.bfloat16), _randn(g, 128)
    mean, rstd, y = torch.empty(5000, device=DEV), torch.empty(5000, device=DEV), torch.empty_like(x)
    dsa.dsa_layernorm(x, w, None, 1e-6, y, mean, rstd)
    need = dsa.layernorm_bwd_workspace(5000, 128)
    wss = [dsa.alloc_workspace(c["shape"], dsa.DSA_OP_DENSE_ATTN) for c in cases]
    nws = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in cases]

    def step(i):
        o, l = _dense(cases[i], ws=wss[i])
        dx, dw, db = torch.empty_like(x), torch.empty(128, device=DEV), torch.empty(128, device=DEV)
        dsa.dsa_layernorm_bwd(dy, x, w, mean, rstd, dx, dw, db, nws[i], need)
        return o, l, dx, dw, db

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = [None, None]
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(i)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    dsa.dsa_check()


# ------------------------------------------------------------------ together

def test_serving_step_append_then_attend():
    """Decode steps: every new token is appended and attended at once, dense
    while the context fits topk, and dsa_forward over the same caches selects
    all keys there and gives the same attention."""
    g = _gen(21)
    B, room, page, H = 3, 512, 128, 128
    ca = _cache(B, room, page, 128, 576, 21)
    ca["kv"].fill_(math.nan)
    shape = dsa.DsaShape(B, 1, room, 64, 128, 512, H, 576, 512, 1.0 / 24)
    rk = dsa.rope_spec(64)
    rc = dsa.rope_spec(64, rot_begin=512, layout=dsa.DSA_ROPE_INTERLEAVED)
    fill = dsa.DsaShape(B, 200, room, 64, 128, 512, H, 576, 512, 1.0 / 24)
    k, c = _randn(g, B, 200, 128, dtype=torch.bfloat16), _randn(g, B, 200, 576, dtype=torch.bfloat16)
    lens = torch.tensor([200, 1, 127], dtype=torch.int32, device=DEV)
    dsa.dsa_cache_append(fill, k, None, None, 1e-6, rk, c, rc, None, lens, ca["codes"], ca["scale"], ca["kv"],
                         layout=ca["layout"])
    ws = dsa.alloc_workspace(shape, dsa.DSA_OP_DENSE_ATTN)
    fws = dsa.alloc_workspace(shape, dsa.DSA_OP_FORWARD)
    for step in range(3):
        k1, c1 = _randn(g, B, 1, 128, dtype=torch.bfloat16), _randn(g, B, 1, 576, dtype=torch.bfloat16)
        q = _randn(g, B, 1, H, 576, dtype=torch.bfloat16)
        dsa.dsa_cache_append(shape, k1, None, None, 1e-6, rk, c1, rc, lens, None, ca["codes"], ca["scale"],
                             ca["kv"], layout=ca["layout"])
        dsa.dsa_rope(dsa.rope_spec(64, rot_begin=512, layout=dsa.DSA_ROPE_INTERLEAVED), q, q, q_pos0=lens)
        now = lens + 1
        out, lse = torch.empty(B, 1, H, 512, device=DEV), torch.empty(B, 1, H, device=DEV)
        dsa.dsa_dense_attn(shape, q, ca["kv"], lens, now, out, lse, *ws, layout=ca["layout"])
        case = {"shape": shape, "q": q, "kv": ca["kv"], "rows": ca["rows"]}
        seen = [[int(n)] for n in now]
        _check_dense(case, out, lse, seen)
        iq = _randn(g, B, 1, 64, 128, dtype=torch.bfloat16)
        dsa.dsa_rope(rk, iq, iq, q_pos0=lens)
        codes, scale = torch.empty(B, 1, 64, 128, dtype=torch.uint8, device=DEV), torch.empty(B, 1, 64, device=DEV)
        dsa.dsa_quantize_e4m3(iq, codes, scale)
        idx = torch.empty(B, 1, 512, dtype=torch.int32, device=DEV)
        out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
        dsa.dsa_forward(shape, codes, scale, _randn(g, B, 1, 64), ca["codes"], ca["scale"], lens, now, q,
                        ca["kv"], idx, out2, lse2, *fws, layout=ca["layout"])
        dsa.dsa_check()
        for b, (n,) in enumerate(seen):
            assert sorted(i for i in idx[b, 0].tolist() if i >= 0) == list(range(n))
        _check_dense(case, out2, lse2, seen)
        lens = now


def test_decode_step_in_a_graph_on_another_stream():
    """append -> rotate -> dense attention captured once and replayed as the
    sequences grow; the same calls made one by one give the same bits."""
    g = _gen(31)
    B, room, H = 2, 256, 16
    shape = dsa.DsaShape(B, 1, room, 64, 128, 512, H, 576, 512, 1.0 / 24)
    rk, rc = dsa.rope_spec(64), dsa.rope_spec(64, rot_begin=512, layout=dsa.DSA_ROPE_INTERLEAVED)
    ca, cb = _cache(B, room, 128, 128, 576, 31), _cache(B, room, 128, 128, 576, 31)
    for c in (ca, cb):
        c["kv"].fill_(math.nan)
    pos, now = torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
    k, c1 = torch.empty(B, 1, 128, device=DEV, dtype=torch.bfloat16), torch.empty(B, 1, 576, device=DEV, dtype=torch.bfloat16)
    q = torch.empty(B, 1, H, 576, device=DEV, dtype=torch.bfloat16)
    ws = [dsa.alloc_workspace(shape, dsa.DSA_OP_DENSE_ATTN) for _ in range(2)]

    def step(ca, q, turned, out, lse, ws):
        dsa.dsa_cache_append(shape, k, None, None, 1e-6, rk, c1, rc, pos, None, ca["codes"], ca["scale"], ca["kv"],
                             layout=ca["layout"])
        dsa.dsa_rope(rc, q, turned, q_pos0=pos)
        dsa.dsa_dense_attn(shape, turned, ca["kv"], pos, now, out, lse, *ws, layout=ca["layout"])

    def bufs():
        return torch.empty_like(q), torch.empty(B, 1, H, 512, device=DEV), torch.empty(B, 1, H, device=DEV)
    ta, tb = bufs(), bufs()
    for t in (k, c1, q):
        t.copy_(_randn(g, *t.shape))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(ca, q, *ta, ws[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step(ca, q, *ta, ws[0])
    torch.cuda.current_stream().wait_stream(st)
    for i in range(140):
        for t in (k, c1, q):
            t.copy_(_randn(g, *t.shape))
        pos.fill_(i)
        now.fill_(i + 1)
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            graph.replay()
        step(cb, q, *tb, ws[1])                          # meanwhile, eagerly, on its own cache and workspace
        torch.cuda.current_stream().wait_stream(st)
        for x, y in zip(ta, tb):
            assert torch.equal(x, y), i
    dsa.dsa_check()
    case = {"shape": shape, "q": ta[0], "kv": ca["kv"], "rows": ca["rows"]}
    _check_dense(case, ta[1], ta[2], [[140]] * B)


def test_training_step_of_the_indexer_key():
    """k -> layer norm -> rotation -> FP8 -> warm-up loss, and the loss's dk
    back through rotation and norm: against the chain's gradient in 64 bits on
    the loss's own dk, and against the loss's change along it."""
    g = _gen(22)
    cfg = dsa.custom_config("tiny", n_q=96, n_kv=96, topk=16)
    inp = {n: (t.to(DEV) if torch.is_tensor(t) else t) for n, t in dsa.make_inputs(cfg, seed=5).items()}
    S, D = 96, cfg.idx_dim
    k, w, b = _randn(g, S, D, dtype=torch.bfloat16), 1 + 0.1 * _randn(g, D), 0.1 * _randn(g, D)
    spec = dsa.rope_spec(16, rot_begin=8, amplitude=1.05)
    y, mean, rstd = torch.empty(S, D, device=DEV), torch.empty(S, device=DEV), torch.empty(S, device=DEV)
    dsa.dsa_layernorm(k, w, b, 1e-6, y, mean, rstd)
    turned = torch.empty(1, S, 1, D, device=DEV)
    dsa.dsa_rope(spec, y.view(1, S, 1, D), turned)
    codes, scale = torch.empty(1, S, D, dtype=torch.uint8, device=DEV), torch.empty(1, S, device=DEV)
    dsa.dsa_quantize_e4m3(turned.view(1, S, D).bfloat16(), codes, scale)
    res = dsa.indexer_kl({**inp, "k_fp8": codes, "k_scale": scale}, cfg)
    dsa.dsa_check()
    dk = res["dk"].view(1, S, 1, D)
    dy = torch.empty_like(dk)
    dsa.dsa_rope(spec, dk, dy, backward=True)
    n = dsa.layernorm_bwd_workspace(S, D)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    dx, dw, db = torch.empty(S, D, device=DEV), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    dsa.dsa_layernorm_bwd(dy.view(S, D), k, w, mean, rstd, dx, dw, db, ws, n)
    # 64-bit chain through autograd
    k64, w64, b64 = (t.double().requires_grad_() for t in (k, w, b))
    m = k64.mean(-1, keepdim=True)
    hat = (k64 - m) / ((k64 - m).square().mean(-1, keepdim=True) + 1e-6).sqrt()
    f = torch.tensor(list(spec.freq[:8]), dtype=torch.float64, device=DEV)
    a = torch.arange(S, device=DEV).double()[:, None] * f
    z = hat * w64 + b64
    u, v = z[:, 8:16], z[:, 16:24]
    c, s = a.cos() * spec.amplitude, a.sin() * spec.amplitude
    t = torch.cat([z[:, :8], u * c - v * s, u * s + v * c, z[:, 24:]], -1)
    (t * res["dk"].view(S, D).double()).sum().backward()
    # dx: 72 + 20 roundings of the row's largest gradient times w, rstd and the
    # pair's amplitude; dweight, dbias: of the column's sum of sizes
    top = res["dk"].view(S, D).double().abs().amax(-1, keepdim=True) * 2.2 * float(w.abs().max())
    r = rstd.double()[:, None]
    _within(dx, k64.grad, r * top * (2 + hat.detach().abs() * float(hat.detach().abs().max())) * 92 * U, "dx")
    _within(dw, w64.grad, (top * hat.detach().abs()).sum(0) * 92 * U, "dweight")
    _within(db, b64.grad, top.expand(S, D).sum(0) * 92 * U, "dbias")
