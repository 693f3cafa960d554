"""Refusals of the operators next to the sparse path (rotary positions, layer
norm, cache append, dense attention), and the frequencies dsa_rope_init fills
in. No GPU: every case ends in the argument checks."""
import ctypes
import math

import pytest

import sparse_attention_long_fp8_b200 as dsa
from sparse_attention_long_fp8_b200 import build as dsa_build

FAKE = 0x100000      # never dereferenced: validation fails before any launch


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load_library()


def _spec(**kw):
    return dsa.rope_spec(kw.pop("rot_dim", 64), **kw)


# ------------------------------------------------------------------ frequencies

@pytest.mark.parametrize("rot", [2, 6, 64, 256])
def test_plain_frequencies(lib, rot):
    s = _spec(rot_dim=rot, base=10000.0)
    for i in range(rot // 2):
        assert s.freq[i] == pytest.approx(math.exp(-2.0 * i / rot * math.log(10000.0)), rel=1e-14)
    assert s.amplitude == 1.0 and s.rot_begin == 0


def test_linear_frequencies_divide_by_the_factor(lib):
    a, b = _spec(), _spec(scaling=dsa.DSA_ROPE_LINEAR, factor=8.0)
    for i in range(32):
        assert b.freq[i] == pytest.approx(a.freq[i] / 8.0, rel=1e-15)


def test_yarn_keeps_fast_pairs_and_divides_slow_ones(lib):
    L, s, fast, slow = 4096, 16.0, 32.0, 1.0
    a = _spec()
    y = _spec(scaling=dsa.DSA_ROPE_YARN, factor=s, orig_context=L, beta_fast=fast, beta_slow=slow)
    kinds = set()
    for i in range(32):
        turns = L * a.freq[i] / (2 * math.pi)
        if turns >= fast:
            kinds.add("fast")
            assert y.freq[i] == a.freq[i]
        elif turns <= slow:
            kinds.add("slow")
            assert y.freq[i] == pytest.approx(a.freq[i] / s, rel=1e-15)
        else:
            kinds.add("between")
            assert a.freq[i] / s < y.freq[i] < a.freq[i]
            g = (turns - slow) / (fast - slow)
            assert y.freq[i] == pytest.approx(a.freq[i] * (1 - g) / s + a.freq[i] * g, rel=1e-13)
    assert kinds == {"fast", "between", "slow"}


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(rot_begin=-1), dict(layout=2),
    dict(base=0.0), dict(base=math.inf), dict(scaling=3), dict(amplitude=math.nan),
    dict(scaling=dsa.DSA_ROPE_LINEAR, factor=0.0),
    dict(scaling=dsa.DSA_ROPE_YARN, factor=2.0, orig_context=0),
    dict(scaling=dsa.DSA_ROPE_YARN, factor=2.0, orig_context=10, beta_fast=1.0, beta_slow=1.0)])
def test_rope_init_refuses(lib, kw):
    with pytest.raises(dsa.DsaError) as e:
        _spec(**kw)
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG


# ------------------------------------------------------------------ rotary positions

def _rope(lib, spec=None, x=FAKE, out=FAKE, size=(2, 3, 4, 128), dtype=dsa.DSA_BF16, xs=None, os_=None):
    B, T, H, D = size
    dense = (T * H * D, H * D, D)
    v = dsa.DsaRopeView(B, T, H, D, dtype, xs or dense, os_ or dense)
    return lib.dsa_rope(ctypes.byref(spec or _spec()), ctypes.byref(v), x, out, None, None, 0, None)


def test_rope_refuses_bad_arguments(lib):
    bad = dsa.DSA_ERR_INVALID_ARG
    assert _rope(lib, x=None) == bad
    assert _rope(lib, x=FAKE + 1) == bad
    assert _rope(lib, dtype=7) == bad
    assert _rope(lib, size=(0, 3, 4, 128)) == bad
    assert _rope(lib, size=(1 << 15, 1 << 15, 4, 128)) == bad
    assert _rope(lib, spec=_spec(rot_begin=65)) == bad                 # 65 + 64 > 128
    assert _rope(lib, size=(2, 3, 4, 63)) == bad
    assert _rope(lib, xs=(-1, 512, 128)) == bad
    s = _spec()
    s.freq[5] = math.inf
    assert _rope(lib, spec=s) == bad
    v = dsa.DsaRopeView(1, 1, 1, 64, 1, (64, 64, 64), (64, 64, 64))
    assert lib.dsa_rope(None, ctypes.byref(v), FAKE, FAKE, None, None, 0, None) == bad
    assert lib.dsa_rope(ctypes.byref(s), None, FAKE, FAKE, None, None, 0, None) == bad


def test_rope_refuses_overlap(lib):
    bad, none = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_NO_DEVICE
    dense = (3 * 4 * 128, 4 * 128, 128)
    assert _rope(lib, out=FAKE + 2) == bad                             # shifted by one element
    assert _rope(lib, os_=(0, 512, 128)) == bad                        # rows written twice
    assert _rope(lib, os_=(3 * 4 * 128, 4 * 128, 64)) == bad           # rows overlap
    assert _rope(lib, xs=dense, os_=(4096, 4 * 128, 128)) == bad       # same start, other strides
    # slices of one wider buffer: dims 0..63 into 64..127 are apart, into 32..95 not
    import torch
    if torch.cuda.is_available():
        pytest.skip("the accepted forms are launched by the GPU tests")
    wide = (3 * 4 * 128, 4 * 128, 128)
    assert _rope(lib, size=(2, 3, 4, 64), xs=wide, os_=wide, out=FAKE + 128) == none
    assert _rope(lib, size=(2, 3, 4, 64), xs=wide, os_=wide, out=FAKE + 64) == bad
    # a broadcast x is read, never written
    assert _rope(lib, xs=(0, 512, 128), out=FAKE + (1 << 20)) == none


# ------------------------------------------------------------------ layer norm

def _norm(lib, rows=4, dim=128, x=FAKE, xd=dsa.DSA_BF16, xs=128, y=FAKE + (1 << 20), yd=dsa.DSA_BF16,
          ys=128, eps=1e-6):
    return lib.dsa_layernorm(rows, dim, x, xd, xs, None, None, eps, y, yd, ys, None, None, None)


def test_layernorm_refuses(lib):
    bad = dsa.DSA_ERR_INVALID_ARG
    assert _norm(lib, rows=-1) == bad
    assert _norm(lib, dim=0) == bad
    assert _norm(lib, dim=16385, xs=16385, ys=16385) == dsa.DSA_ERR_UNSUPPORTED
    assert _norm(lib, x=None) == bad
    assert _norm(lib, xd=2) == bad
    assert _norm(lib, ys=127) == bad
    assert _norm(lib, eps=-1.0) == bad
    assert _norm(lib, eps=math.nan) == bad
    assert _norm(lib, x=FAKE + 1) == bad
    assert _norm(lib, y=FAKE + 2) == bad                # overlaps x
    assert _norm(lib, y=FAKE, yd=dsa.DSA_F32) == bad    # the same start, another dtype
    assert _norm(lib, rows=0) == dsa.DSA_OK


def _norm_bwd(lib, rows=4, dim=128, dy=FAKE, x=FAKE + (1 << 20), dx=FAKE + (2 << 20), mean=FAKE + (3 << 20),
              dw=FAKE + (4 << 20), ws=FAKE + (5 << 20), n=1 << 30):
    b = dsa.DSA_BF16
    return lib.dsa_layernorm_bwd(rows, dim, dy, b, dim, x, b, dim, None, mean, mean, dx, b, dim, dw, None,
                                 ws, n, None)


def test_layernorm_bwd_refuses(lib):
    bad = dsa.DSA_ERR_INVALID_ARG
    assert _norm_bwd(lib, dim=0) == bad
    assert _norm_bwd(lib, mean=None) == bad
    assert _norm_bwd(lib, dy=None) == bad
    assert _norm_bwd(lib, dx=FAKE + 2) == bad
    assert _norm_bwd(lib, dx=FAKE + (1 << 20) + 2) == bad
    assert _norm_bwd(lib, n=16) == dsa.DSA_ERR_WORKSPACE
    assert _norm_bwd(lib, ws=None) == dsa.DSA_ERR_WORKSPACE
    assert _norm_bwd(lib, ws=FAKE + 4) == bad
    assert _norm_bwd(lib, dim=20000) == dsa.DSA_ERR_UNSUPPORTED
    assert dsa.layernorm_bwd_workspace(0, 128) == 0
    assert dsa.layernorm_bwd_workspace(1, 128) == 2 * 128 * 4
    with pytest.raises(dsa.DsaError):
        dsa.layernorm_bwd_workspace(-1, 128)


# ------------------------------------------------------------------ cache append

def _append(lib, shape=None, layout=None, k=FAKE, c=FAKE, kv=FAKE, idx=None, lat=None, eps=1e-6):
    s = shape or dsa.DsaShape(2, 1, 256, 64, 128, 2048, 128, 576, 512, 1.0)
    return lib.dsa_cache_append(ctypes.byref(s), ctypes.byref(layout) if layout else None, k, None, None,
                                eps, ctypes.byref(idx or _spec()), c,
                                ctypes.byref(lat or _spec(rot_begin=512)), None, None, FAKE, FAKE, kv, None)


def test_append_refuses(lib):
    bad = dsa.DSA_ERR_INVALID_ARG
    assert _append(lib, k=None) == bad
    assert _append(lib, k=FAKE + 4) == bad
    assert _append(lib, c=FAKE + 8) == bad
    assert _append(lib, eps=-1.0) == bad
    assert _append(lib, idx=_spec(rot_begin=66)) == bad
    assert _append(lib, lat=_spec(rot_begin=514)) == bad
    assert _append(lib, dsa.DsaShape(2, 1, 256, 64, 64, 2048, 128, 576, 512, 1.0)) == dsa.DSA_ERR_UNSUPPORTED
    assert _append(lib, dsa.DsaShape(2, 1, 256, 64, 128, 2048, 128, 512, 512, 1.0)) == dsa.DSA_ERR_UNSUPPORTED
    assert _append(lib, dsa.DsaShape(0, 1, 256, 64, 128, 2048, 128, 576, 512, 1.0)) == bad
    lay = dsa.DsaLayout()
    lay.row_pos = FAKE
    assert _append(lib, layout=lay) == bad
    lay = dsa.DsaLayout()
    lay.block_table, lay.max_pages, lay.page_size, lay.pool_rows = FAKE, 1, 128, 1024
    assert _append(lib, layout=lay) == bad              # 256 keys need two pages
    lay.max_pages, lay.page_size = 4, 96
    assert _append(lib, layout=lay) == bad


# ------------------------------------------------------------------ dense attention

def _dense(lib, q=FAKE, kv=FAKE, out=FAKE, ws=FAKE, n=1 << 40, layout=None, dtype=1, **kw):
    f = dict(batch=2, n_q=1, n_kv=256, idx_heads=0, idx_dim=0, topk=0, heads=128, qk_dim=576, v_dim=512,
             softmax_scale=0.04)
    f.update(kw)
    s = dsa.DsaShape(*f.values())
    return lib.dsa_dense_attn_ex(ctypes.byref(s), ctypes.byref(layout) if layout else None, q, kv, None, None,
                                 out, dtype, None, ws, n, None)


def test_dense_refuses(lib):
    bad, uns = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    assert _dense(lib, q=None) == bad
    assert _dense(lib, kv=FAKE + 8) == bad
    assert _dense(lib, dtype=2) == bad
    assert _dense(lib, heads=0) == uns
    assert _dense(lib, heads=129) == uns
    assert _dense(lib, qk_dim=64, v_dim=64) == uns
    assert _dense(lib, batch=1 << 12, n_q=17) == uns
    assert _dense(lib, n_kv=0) == bad
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert _dense(lib, softmax_scale=scale) == bad
    assert _dense(lib, ws=None) == dsa.DSA_ERR_WORKSPACE
    assert _dense(lib, n=1024) == dsa.DSA_ERR_WORKSPACE
    assert _dense(lib, ws=FAKE + 128) == bad


def test_dense_workspace_does_not_depend_on_lengths(lib):
    def size(**kw):
        f = dict(batch=1, n_q=1, n_kv=64, idx_heads=0, idx_dim=0, topk=0, heads=128, qk_dim=576,
                 v_dim=512, softmax_scale=0.04)
        f.update(kw)
        return dsa.workspace_size(dsa.DsaShape(*f.values()), dsa.DSA_OP_DENSE_ATTN)
    assert size() == size(batch=64, n_kv=65536) == size(n_q=4, n_kv=1)
    assert size(heads=1) < size()


# ------------------------------------------------------------------ the Python binding

def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    import torch
    x = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError):
        dsa.dsa_rope(_spec(), x, x)                                  # CPU
    with pytest.raises(ValueError):
        dsa.dsa_rope(_spec(), x, torch.zeros(1, 2, 3, 63))
    with pytest.raises(ValueError):
        dsa.dsa_rope(_spec(), x, x.bfloat16())
    with pytest.raises(ValueError):
        dsa.dsa_rope(_spec(), x, x, q_pos0=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        dsa.dsa_rope(_spec(), x.half(), x.half())
    with pytest.raises(ValueError):
        dsa.dsa_rope(_spec(), x.transpose(2, 3), x.transpose(2, 3))
    y = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        dsa.dsa_layernorm(y, None, None, 1e-6, y)                     # CPU
    with pytest.raises(ValueError):
        dsa.dsa_layernorm(y, torch.zeros(7), None, 1e-6, y)
    with pytest.raises(ValueError):
        dsa.dsa_layernorm(y.t(), None, None, 1e-6, y.t())
    with pytest.raises(ValueError):
        dsa.dsa_layernorm_bwd(y, y, None, torch.zeros(3), torch.zeros(4), y)
    s = dsa.DsaShape(1, 1, 4, 64, 128, 1, 128, 576, 512, 1.0)
    q, kv = torch.zeros(1, 1, 128, 576).bfloat16(), torch.zeros(4, 576).bfloat16()
    with pytest.raises(ValueError):
        dsa.dsa_dense_attn(s, q, kv, None, None, torch.zeros(1, 1, 128, 512))   # CPU
    with pytest.raises(ValueError):
        dsa.dsa_dense_attn(s, q, kv[:3], None, None, torch.zeros(1, 1, 128, 512))


def test_binding_refuses_a_workspace_shorter_than_it_is_said_to_be(lib):
    import torch
    s = dsa.DsaShape(1, 1, 4, 64, 128, 1, 128, 576, 512, 1.0)
    q, kv = torch.zeros(1, 1, 128, 576).bfloat16(), torch.zeros(4, 576).bfloat16()
    out, ws = torch.zeros(1, 1, 128, 512), torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError, match="1024 bytes, ws_bytes is 1025"):
        dsa.dsa_dense_attn(s, q, kv, None, None, out, ws=ws, ws_bytes=1025)
    y, m = torch.zeros(4, 8), torch.zeros(4)
    with pytest.raises(ValueError, match="1024 bytes, ws_bytes is 2048"):
        dsa.dsa_layernorm_bwd(y, y, None, m, m, y, torch.zeros(8), torch.zeros(8), ws=ws, ws_bytes=2048)


# ------------------------------------------------------------------ spans

def test_spans_that_would_overflow_are_refused(lib):
    bad, big = dsa.DSA_ERR_INVALID_ARG, 1 << 30
    huge = (big, big, 4, 128)                                          # 2^62 rows
    assert _rope(lib, size=huge) == bad
    assert _rope(lib, size=(1 << 20, 3, 4, 128), xs=(1 << 40, 512, 128)) == bad
    assert _norm(lib, rows=1 << 40, xs=1 << 40, ys=1 << 40) == bad
    assert _norm(lib, rows=1 << 20, xs=1 << 30) == bad


def test_layernorm_takes_columns_of_one_buffer_side_by_side(lib):
    import torch
    bad, none = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_NO_DEVICE
    assert _norm(lib, xs=256, ys=256, y=FAKE + 2 * 127) == bad         # one column in common
    assert _norm(lib, xs=256, ys=256, y=FAKE + 2 * 129) == bad         # the last one and the next row's first
    assert _norm(lib, xs=512, ys=256, y=FAKE + 2 * 128) == bad         # other steps
    if torch.cuda.is_available():
        pytest.skip("the accepted forms are launched by the GPU tests")
    assert _norm(lib, xs=256, ys=256, y=FAKE + 2 * 128) == none
    assert _norm(lib, xs=384, ys=192, yd=dsa.DSA_F32, y=FAKE + 2 * 128) == none
