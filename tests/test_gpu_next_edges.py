"""Edges of the operators next to the sparse path: rows of a few values, values
that are not finite, positions far out. Tolerances count roundings as in
test_gpu_next.py."""
import math
import random
from fractions import Fraction

import pytest
import torch

import sparse_attention_long_fp8_b200 as dsa
from test_gpu_next import (DEV, HALF, U, _cache, _check_dense, _clean, _dense, _dense_case, _gen,  # noqa: F401
                           _norm64, _randn, _rope_tol, _turn64, _within)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ layer norm

@pytest.mark.parametrize("xt,gt,dt", [(torch.bfloat16, torch.float32, torch.bfloat16),
                                      (torch.float32, torch.float32, torch.float32),
                                      (torch.float32, torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("rows", [1, 3, 257, 90001])
@pytest.mark.parametrize("dim", [1, 2, 3, 4])
def test_layernorm_gradient_of_rows_of_a_few_values(dim, rows, xt, gt, dt):
    """dx of rows of two values is a millionth of its terms (1 - hat^2 = eps
    rstd^2): it has to be right relative to itself."""
    g = _gen(rows * 5 + dim)
    wide = (_randn(g, rows, dim + 3) * 2 + 0.5).to(xt)
    x, dy, w = wide[:, 1:1 + dim], _randn(g, rows, dim, dtype=gt), 1 + 0.2 * _randn(g, dim)
    m, r, _ = _norm64(x, 1e-6)
    mean, rstd = m[:, 0].float(), r[:, 0].float()
    n = dsa.layernorm_bwd_workspace(rows, dim)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    hat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    d = dy.double()
    for weight in (w, None):
        dx = torch.empty(rows, dim, device=DEV, dtype=dt)
        dw, db = torch.full((dim,), 9.0, device=DEV), torch.full((dim,), 9.0, device=DEV)
        dsa.dsa_layernorm_bwd(dy, x, weight, mean, rstd, dx, dw, db, ws, n)
        q = d * (weight.double() if weight is not None else 1.0)
        want = rstd.double()[:, None] * (q - q.mean(-1, keepdim=True) - hat * (q * hat).mean(-1, keepdim=True))
        size = rstd.double()[:, None] * (q.abs() + q.abs().mean(-1, keepdim=True)
                                         + hat.abs() * (q * hat).abs().mean(-1, keepdim=True))
        # at most 16 roundings of 2^-53 on either side; one to fp32, one to dx's type
        lost = size * 32 * 2.0 ** -53
        _within(dx, want, lost + (want.abs() + lost) * (HALF[dt] + 2 * U), "dx")
        # fp64 within a CTA; at most 352 partial rows, 11 in a thread and 32 + 5 sums after that
        _within(dw, (d * hat).sum(0), (d * hat).abs().sum(0) * 64 * U, "dweight")
        _within(db, d.sum(0), d.abs().sum(0) * 64 * U, "dbias")
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    dsa.dsa_layernorm_bwd(dy, x, None, mean, rstd, dx2, dw2, db2, ws, n)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)      # the same bits
    if dt == gt:
        a = dy.clone()
        dsa.dsa_layernorm_bwd(a, x, None, mean, rstd, a)                               # in place
        assert torch.equal(a, dx)


@pytest.mark.parametrize("dim", [5, 37, 129, 200, 1000, 1001, 1032, 2056, 4097, 9000])
def test_layernorm_gradient_of_large_constant_rows(dim):
    """Equal values of 1e36: hat is 0, but mean * rstd is past fp32, so places
    past the row's end must not form it."""
    g = _gen(dim)
    rows = 7
    x = torch.full((rows, dim), 1e36, device=DEV)
    dy, w = _randn(g, rows, dim), _randn(g, dim)
    mean, rstd = x[:, 0].clone(), torch.full((rows,), 1000.0, device=DEV)      # eps = 1e-6
    n = dsa.layernorm_bwd_workspace(rows, dim)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    dx, dw, db = torch.empty_like(x), torch.empty(dim, device=DEV), torch.empty(dim, device=DEV)
    dsa.dsa_layernorm_bwd(dy, x, w, mean, rstd, dx, dw, db, ws, n)
    q = dy.double() * w.double()
    want = 1000.0 * (q - q.mean(-1, keepdim=True))
    _within(dx, want, 1000.0 * (q.abs() + q.abs().mean(-1, keepdim=True)) * 73 * U, "dx")
    assert (dw == 0).all()
    _within(db, dy.double().sum(0), dy.double().abs().sum(0) * 64 * U, "dbias")


# ------------------------------------------------------------------ dense attention

@pytest.mark.parametrize("n", [1, 5, 31, 32, 33, 63, 64, 127, 128, 129, 160, 1153, 9473])
def test_dense_nan_query(n):
    """Every key's logit is NaN, whole rows and cut ones: out and lse are NaN, and
    the heads beside it are as without it."""
    c = _dense_case([n, 200], 1, 16, 128, n)
    want, wlse = _dense(c)
    for dim in (3, 570):
        q = c["q"].clone()
        q[0, 0, 2, dim] = math.nan
        out, lse = _dense({**c, "q": q}, torch.float32)
        assert out[0, 0, 2].isnan().all() and lse[0, 0, 2].isnan()
        rest = [h for h in range(16) if h != 2]
        assert torch.equal(out[0, 0, rest].bfloat16(), want[0, 0, rest]) and torch.equal(lse[0, 0, rest], wlse[0, 0, rest])
        assert torch.equal(out[1].bfloat16(), want[1]) and torch.equal(lse[1], wlse[1])
    dsa.dsa_check()


@pytest.mark.parametrize("n", [1, 2, 33, 100, 129, 130, 1153, 9473])
@pytest.mark.parametrize("dim", [0, 570])
def test_dense_nan_in_one_key(n, dim):
    """A visible key with NaN, in its value dims or only in its rotated ones, makes
    its row NaN wherever it lies and the row is cut; behind the row it changes nothing."""
    c = _dense_case([n, 77], 1, 40, 128, n + 1, room=n + 130)
    want = _dense(c)
    for at in sorted({0, n // 2, n - 1}):
        kv = c["kv"].clone()
        kv[c["rows"][0, at], dim] = math.nan
        out, lse = _dense({**c, "kv": kv})
        assert out[0].isnan().all() and lse[0].isnan().all(), at
        assert torch.equal(out[1], want[0][1]) and torch.equal(lse[1], want[1][1])


@pytest.mark.parametrize("n", [1, 20, 40, 300, 5000])
def test_dense_logits_of_minus_infinity(n):
    """Keys at minus infinity have no weight; NaN beside them still shows."""
    c = _dense_case([n], 1, 8, 128, n + 2)
    kv, q = c["kv"].clone(), c["q"].clone()
    q[..., 575] = 1.0
    kv[c["rows"][0, :n], 575] = -math.inf
    out, lse = _dense({**c, "kv": kv, "q": q})
    assert (out == 0).all() and (lse == -math.inf).all()             # as a row that sees no key
    kv[c["rows"][0, n - 1], 574] = math.nan
    out, lse = _dense({**c, "kv": kv, "q": q})
    assert out.isnan().all() and lse.isnan().all()
    if n > 1:                                                        # only the first key counts
        kv = c["kv"].clone()
        kv[c["rows"][0, 1:n], 575] = -math.inf
        out, lse = _dense({**c, "kv": kv, "q": q}, torch.float32)
        one = {**c, "kv": kv, "q": q}
        _check_dense(one, out, lse, [[1]])


# ------------------------------------------------------------------ cache append

def _append(k, w, b, rk, idx, page=128):
    """One token per sequence at position 5 of fresh caches: codes (as values),
    scales, latent rows, in the sequences' order."""
    B = k.shape[0]
    ca = _cache(B, 256, page, idx, 64, 3)
    shape = dsa.DsaShape(B, 1, 256, 64, idx, 2048, 128, 64, 64, 1.0)
    c = torch.ones(B, 1, 64, device=DEV, dtype=torch.bfloat16)
    dsa.dsa_cache_append(shape, k, w, b, 1e-6, rk, c, dsa.rope_spec(8), torch.full((B,), 5, dtype=torch.int32, device=DEV),
                         None, ca["codes"], ca["scale"], ca["kv"], layout=ca["layout"])
    dsa.dsa_check()
    at = ca["rows"][:, 5]
    return ca["codes"][at].view(torch.float8_e4m3fn).float(), ca["scale"][at], ca["kv"][at]


@pytest.mark.parametrize("idx", [32, 128])
@pytest.mark.parametrize("layout", [dsa.DSA_ROPE_HALF, dsa.DSA_ROPE_INTERLEAVED])
@pytest.mark.parametrize("rot,begin", [(8, 0), (8, 16), (6, 3)])
def test_append_keys_that_are_not_finite(rot, begin, layout, idx):
    g = _gen(idx + rot)
    B, rk = 6, dsa.rope_spec(rot, rot_begin=begin, layout=layout)
    k = _randn(g, B, 1, idx, dtype=torch.bfloat16)
    want = _append(k, None, None, rk, idx)
    assert want[0].isfinite().all()
    bad = k.clone()
    bad[0, 0, 0] = bad[1, 0, idx - 1] = bad[2, 0, begin] = math.nan
    bad[3, 0, 7], bad[4, 0, idx // 2] = math.inf, -math.inf
    codes, scale, kv = _append(bad, None, None, rk, idx)
    # the norm spreads NaN and infinity over the whole key: NaN codes, scale 1
    assert codes[:5].isnan().all() and (scale[:5] == 1.0).all()
    assert torch.equal(codes[5], want[0][5]) and scale[5] == want[1][5] and torch.equal(kv, want[2])
    # a bias that is not finite: only its own dim, outside the rotated part, is
    b = torch.zeros(idx, device=DEV)
    b[idx - 2] = math.nan
    rest = [i for i in range(idx) if i != idx - 2]
    codes, scale, _ = _append(k, None, b, rk, idx)
    assert codes[:, idx - 2].isnan().all() and (scale == 1.0).all()
    # the other values against scale 1: half a step of e4m3, 2^-4 of the value, 2^-10 below 2^-6
    was = (want[0] * want[1][:, None])[:, rest]
    step = torch.maximum(was.abs() * 2.0 ** -4, torch.full_like(was, 2.0 ** -10))
    # `was` itself is off by half a step of its own code
    own = torch.maximum(was.abs() * 2.0 ** -4, want[1][:, None] * 2.0 ** -10)
    assert ((codes[:, rest] - was).abs() <= (step + own) * 1.07).all()
    b[idx - 2] = math.inf
    codes, scale, _ = _append(k, None, b, rk, idx)
    assert (scale == math.inf).all() and codes[:, idx - 2].isnan().all() and (codes[:, rest] == 0).all()


def test_append_nan_key_leaves_the_other_keys_scores_and_choices():
    g = _gen(77)
    n, topk = 300, 64
    shape = dsa.DsaShape(1, n, n, 64, 128, topk, 128, 576, 512, 1.0 / 24)
    one = dsa.DsaShape(1, 1, n, 64, 128, topk, 128, 576, 512, 1.0 / 24)
    rk, rc = dsa.rope_spec(64), dsa.rope_spec(64, rot_begin=512)
    k, c = _randn(g, 1, n, 128, dtype=torch.bfloat16), _randn(g, 1, n, 576, dtype=torch.bfloat16)
    iq, w = _randn(g, 1, 1, 64, 128, dtype=torch.bfloat16), _randn(g, 1, 1, 64).abs()
    qc, qs = torch.empty(1, 1, 64, 128, dtype=torch.uint8, device=DEV), torch.empty(1, 1, 64, device=DEV)
    dsa.dsa_quantize_e4m3(iq, qc, qs)
    pos, lens = torch.tensor([n - 1], dtype=torch.int32, device=DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    got = []
    for bad in (False, True):
        kk = k.clone()
        if bad:
            kk[0, 17, 3] = math.nan
        ca = _cache(1, n, 128, 128, 576, 9)
        dsa.dsa_cache_append(shape, kk, None, None, 1e-6, rk, c, rc, None, None, ca["codes"], ca["scale"], ca["kv"],
                             layout=ca["layout"])
        scores = torch.empty(1, 1, n, device=DEV)
        dsa.dsa_indexer_scores(one, qc, qs, w, ca["codes"], ca["scale"], pos, lens, 0, 1, scores, layout=ca["layout"])
        idx = torch.empty(1, 1, topk, dtype=torch.int32, device=DEV)
        dsa.dsa_indexer_topk(one, qc, qs, w, ca["codes"], ca["scale"], pos, lens, 0, 1, idx, layout=ca["layout"])
        dsa.dsa_check()
        got.append((scores.view(-1), idx.view(-1).tolist()))
    rest = [i for i in range(n) if i != 17]
    assert torch.equal(got[0][0][rest], got[1][0][rest])
    for s, idx in got:
        chosen = [i for i in idx if i != 17]
        assert len(set(idx)) == topk and min(idx) >= 0 and max(idx) < n
        # all but key 17 in the order of their scores
        kth = s[rest].sort(descending=True).values[len(chosen) - 1]
        assert (s[chosen] >= kth).all()


# ------------------------------------------------------------------ rotary positions

# 2 pi to 60 digits
_TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


@pytest.mark.parametrize("layout", [dsa.DSA_ROPE_HALF, dsa.DSA_ROPE_INTERLEAVED])
@pytest.mark.parametrize("back", [False, True])
def test_rope_cos_and_sin_to_an_ulp(layout, back):
    """Pairs (1, 0) turn to (cos, sin) exactly as the kernel forms them, against
    the exact product of position and frequency, reduced exactly."""
    spec = dsa.rope_spec(16, layout=layout)
    rnd = random.Random(5)
    pos = [0, 1, 2, 3, 1000, 65535, 1 << 20, (1 << 27) - 1, (1 << 29) + 7, (1 << 31) - 2]
    pos += [int(2.0 ** rnd.uniform(0, 31)) for _ in range(500)]
    freq = [Fraction(spec.freq[i]) for i in range(8)]
    angle = [[(p * f) - _TWO_PI * round(p * f / _TWO_PI) for f in freq] for p in pos]
    want = torch.tensor([[[math.cos(a), (-1 if back else 1) * math.sin(a)] for a in map(float, r)] for r in angle],
                        dtype=torch.float64, device=DEV)
    x = torch.zeros(1, len(pos), 1, 16, device=DEV)
    first = slice(0, 8) if layout == dsa.DSA_ROPE_HALF else slice(0, 16, 2)
    second = slice(8, 16) if layout == dsa.DSA_ROPE_HALF else slice(1, 16, 2)
    x[..., first] = 1.0
    y = torch.empty_like(x)
    dsa.dsa_rope(spec, x, y, row_pos=torch.tensor([pos], dtype=torch.int32, device=DEV), backward=back)
    got = torch.stack([y[0, :, 0, first], y[0, :, 0, second]], -1)
    # the rest of the angle rounds by half an ulp below 1: 2^-25 = U / 2. sin: its last
    # fma U / 2 (values below 1), the cube's and the series' roundings 4 U of at most
    # 0.617 / 6 of the value: U / 2. cos: its last fma U / 2, the square's U of 0.31, the
    # series' 3 U of 0.31: 1.3 U. Left out of the series: U / 28.
    whole = torch.tensor([[float(p * f) for f in freq] for p in pos], dtype=torch.float64, device=DEV)
    _within(got, want, (2.4 * U + whole * 2.0 ** -52)[..., None], "cos, sin")
