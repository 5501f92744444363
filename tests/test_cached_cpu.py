"""The compressed source cache without a GPU: record sizes and layout, refusals
of the C entry points before anything is launched, refusals of the binding,
and the 64-bit reference that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import cached_reference as ref
from attention_residuals_gb300 import (_lib, attnres_cache_load, attnres_cache_row_bytes, attnres_cache_write,
                                       attnres_cached, attnres_cached_fwd)
from attention_residuals_gb300.build import build
from attention_residuals_gb300.custom_ops import _cache_bytes

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers are only used without a GPU")


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def test_record_bytes(lib):
    for D in list(range(8, 600, 8)) + [1000, 4096, 8192]:
        for bits in (4, 8):
            want = ref.offsets(D, bits)[2]
            assert attnres_cache_row_bytes(D, bits) == want == _cache_bytes(D, bits) and want % 16 == 0
    for D, bits in ((0, 8), (4, 8), (12, 8), (8200, 8), (64, 2), (64, 16), (64, 0)):
        assert lib.attnres_cache_row_bytes(D, bits) == 0
        with pytest.raises(ValueError):
            attnres_cache_row_bytes(D, bits)


def test_params_struct_layout_matches_header():
    P = _lib.AttnresCachedParams
    assert P.N.offset == 16 and P.eps.offset == 24 and P.row_ld.offset == 40 and P.live.offset == 56
    assert P.rows.offset == 64 and ctypes.sizeof(P) == 64 + 8 * _lib.MAX_S


A, B, ODD = 0x100000, 0x900000, 0x100008
ROWS = [  # src, src_ld, N, D, bits, R, ko, rows, row_ld -> status
    ((A, 64, 4, 64, 2, 64, 0, B, 96), 1), ((A, 64, 4, 12, 8, 12, 0, B, 96), 2), ((A, 64, 4, 0, 8, 1, 0, B, 96), 1),
    ((A, 64, 4, 16384, 8, 8, 0, B, 96), 1), ((A, 64, 4, 64, 8, 0, 0, B, 96), 1), ((A, 64, 4, 64, 8, 65, 0, B, 96), 1),
    ((A, 64, 4, 64, 8, 32, 33, B, 96), 1), ((A, 64, 4, 64, 8, 32, -1, B, 96), 1), ((A, 64, -1, 64, 8, 64, 0, B, 96), 1),
    ((A, 56, 4, 64, 8, 64, 0, B, 96), 1), ((A, 68, 4, 64, 8, 64, 0, B, 96), 2), ((ODD, 64, 4, 64, 8, 64, 0, B, 96), 2),
    ((None, 64, 4, 64, 8, 64, 0, B, 96), 1), ((A, 64, 4, 64, 8, 64, 0, None, 96), 1),
    ((A, 64, 4, 64, 8, 64, 0, ODD, 96), 2), ((A, 64, 4, 64, 8, 64, 0, B, 64), 1), ((A, 64, 4, 64, 8, 64, 0, B, 104), 2),
    ((A, 64, 4, 64, 8, 64, 0, A + 256, 96), 1),      # records over the rows they are made from
    ((None, 64, 0, 64, 8, 64, 0, None, 96), 0),      # no tokens: nothing is read
]


@no_gpu
@pytest.mark.parametrize("args,status", ROWS)
def test_write_and_load_refusals(lib, args, status):
    assert lib.attnres_cache_write(*args, None) == status
    src, src_ld, N, D, bits, R, ko, rows, row_ld = args
    if 1 <= R <= D and 0 <= ko <= D - R:
        assert lib.attnres_cache_load(rows, row_ld, N, D, bits, src, src_ld, None) == status


def params(S=3, D=64, R=64, ko=0, N=8, bits=8, ld=None, eps=2.0 ** -23, scale=1.0, norm=0, live=None, live_ld=64,
           rows=0x200000):
    p = _lib.AttnresCachedParams()
    p.S, p.D, p.R, p.key_offset, p.N, p.bits = S, D, R, ko, N, bits
    p.row_ld = 96 if ld is None else ld
    p.eps, p.scale, p.out_norm = eps, scale, norm
    p.live, p.live_ld = live, live_ld
    for s in range(min(max(S, 0), _lib.MAX_S)):
        p.rows[s] = rows + s * 0x10000 if rows else None
    return p


BAD = [
    (dict(S=0), 1), (dict(S=129), 1), (dict(S=128, live=B), 1), (dict(D=12, R=12), 2), (dict(D=8200, R=8), 1),
    (dict(R=0), 1), (dict(R=65), 1), (dict(R=32, ko=33), 1), (dict(ko=-1), 1), (dict(N=-1), 1), (dict(bits=6), 1),
    (dict(ld=64), 1), (dict(ld=100), 2), (dict(norm=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(rows=0), 1), (dict(rows=0x200004), 2), (dict(live=0x900002), 2),
    (dict(live=B, live_ld=32), 1), (dict(live=B, live_ld=68), 2),
]


@no_gpu
@pytest.mark.parametrize("kw,status", BAD)
def test_read_refusals(lib, kw, status):
    p = params(**kw)
    f = 0x500000
    assert lib.attnres_cached_fwd(ctypes.byref(p), f, None, f, f, f, f, None, None) == status
    assert lib.attnres_cached_bwd(ctypes.byref(p), f, None, f, f, f, f, None, None, 64, None, 64, f, None, None, None, f,
                                  1 << 20, None) == status
    assert lib.attnres_cached_bwd_workspace_bytes(ctypes.byref(p)) == 0


@no_gpu
def test_pointer_and_overlap_refusals(lib):
    f = 0x500000
    fwd, bwd = lib.attnres_cached_fwd, lib.attnres_cached_bwd
    p = params()
    assert fwd(None, f, None, f, f, f, f, None, None) == 1
    assert fwd(ctypes.byref(p), None, None, f, f, f, f, None, None) == 1
    assert fwd(ctypes.byref(p), f, None, f + 8, f, f, f, None, None) == 2
    assert fwd(ctypes.byref(p), f, None, f, f + 2, f, f, None, None) == 2
    assert fwd(ctypes.byref(p), f, None, 0x210000 + 64, f, f, f, None, None) == 1   # y over a source's records
    assert fwd(ctypes.byref(params(live=0xa00000)), f, None, 0xa00000 - 512, f, f, f, None, None) == 1
    n = params(norm=1)
    assert fwd(ctypes.byref(n), f, None, f, f, f, f, f, None) == 1           # no weight
    assert fwd(ctypes.byref(n), f, f, f, f, f, f, None, None) == 1           # no o_rstd
    assert fwd(ctypes.byref(n), f, f + 2, f, f, f, f, f, None) == 2

    def back(p, d=None, dld=64, dl=None, dlld=64, dq=f, ws=f, n=1 << 20, dy=f):
        ptrs = None if d is None else (ctypes.c_void_p * 3)(*d)
        return bwd(ctypes.byref(p), f, None, dy, f, f, f, None, ptrs, dld, dl, dlld, dq, None, None, None, ws, n, None)

    far = [0x600000, 0x700000, 0x800000]
    assert back(p, dq=None) == 1 and back(p, dy=f + 2) == 2 and back(p, dy=None) == 1
    assert back(p, dl=0x900000) == 1                                         # a gradient of no live source
    assert back(p, d=[far[0], None, far[2]]) == 1 and back(p, d=[far[0], far[1] + 8, far[2]]) == 2
    assert back(p, d=far, dld=56) == 1 and back(p, d=far, dld=68) == 2
    assert back(p, d=[far[0], far[0] + 512, far[2]]) == 1                    # over another gradient
    assert back(p, d=[far[0], 0x200000 + 64, far[2]]) == 1                   # over the records
    assert back(p, d=[far[0], f + 512, far[2]]) == 1                         # over dy
    lv = params(live=0xa00000)
    assert back(lv, d=far, dl=0xa00000 + 128) == 1                           # over the live source
    assert back(lv, d=far, dl=far[1]) == 1 and back(lv, d=far, dl=0xb00008) == 2


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        attnres_cache_write(x)                                               # no CPU path
    with pytest.raises(TypeError):
        attnres_cache_load(torch.zeros(4, 96, dtype=torch.uint8), 64)
    with pytest.raises(TypeError):
        attnres_cached_fwd(torch.zeros(2, 4, 96, dtype=torch.uint8), torch.zeros(64, dtype=torch.bfloat16), 64)
    with pytest.raises(ValueError):
        attnres_cached_fwd([], torch.zeros(64, dtype=torch.bfloat16), 64)
    with pytest.raises(ValueError):
        attnres_cached([], torch.zeros(64, dtype=torch.bfloat16), 64)
    with pytest.raises(ValueError):
        attnres_cached([torch.zeros(4, 96, dtype=torch.uint8)], torch.zeros(64, dtype=torch.bfloat16), 64, values=[x, x])


@pytest.mark.parametrize("bits", [8, 4])
def test_reference_rounds_to_the_nearest_code(bits):
    """The reference's own rounding against a comparison with every representable value."""
    rng = np.random.RandomState(bits)
    x = torch.from_numpy(rng.randn(64) * 3).bfloat16().double().numpy()
    rec, vals = ref.write_row(x, bits, 64, 0)
    at = ref.offsets(64, bits)[0]
    for g in range(2):
        k = rec[at + g] - 127
        top = np.abs(x[32 * g:32 * g + 32]).max()
        assert top <= ref.GRID[bits][-1] * 2.0 ** k and top > ref.GRID[bits][-1] * 2.0 ** (k - 1)
        grid = np.concatenate([-ref.GRID[bits], ref.GRID[bits]]) * 2.0 ** k
        for i in range(32 * g, 32 * g + 32):
            assert abs(vals[i] - x[i]) == np.abs(grid - x[i]).min()
    if bits == 8:
        codes = torch.frombuffer(bytearray(rec[:64]), dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(codes * 2.0 ** (np.repeat(np.frombuffer(bytes(rec[at:at + 2]), np.uint8), 32) - 127.0), vals)


def test_reference_gradient_against_autograd():
    g = torch.Generator().manual_seed(0)
    S, N, D, R, ko = 3, 5, 24, 10, 7
    v, q, w, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((S, N, D), (R,), (D,), (N, D)))
    for use_w in (True, False):
        a = [t.clone().requires_grad_() for t in (v, q, w)]
        t = a[0][..., ko:ko + R]
        z = 0.5 * (t @ a[1]) / (t.square().mean(-1) + ref.EPS).sqrt()
        o = (torch.softmax(z, 0)[..., None] * a[0]).sum(0)
        y = o / (o.square().mean(-1, keepdim=True) + ref.EPS).sqrt() * a[2] if use_w else o
        grads = torch.autograd.grad(y, a if use_w else a[:2], dy)
        got = ref.read(v.numpy(), q.numpy(), 0.5, ko, w.numpy() if use_w else None, dy.numpy())
        for name, want in zip(("dvalues", "dq_f32", "dw_o_f32"), grads):
            assert np.allclose(got[name][0], want.numpy(), rtol=1e-12, atol=1e-12)
        assert np.allclose(got["y"][0], y.detach().numpy(), rtol=1e-12)
