"""The compressed source cache on the GPU against its definition in 64 bits
(cached_reference.py says where the tolerances come from)."""
import numpy as np
import pytest
import torch

import cached_reference as ref
from attention_residuals_gb300 import (attnres_bwd, attnres_cache_load, attnres_cache_row_bytes, attnres_cache_write,
                                       attnres_cached, attnres_cached_bwd, attnres_cached_fwd,
                                       attnres_check_device_error, attnres_fwd)
from attention_residuals_gb300._lib import AttnresError

pytestmark = pytest.mark.gpu


def rand(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).bfloat16().cuda()


def np64(t):
    return t.detach().double().cpu().numpy()


def sources(S, N, D, bits, R, ko, seed=0):
    """bf16 sources of several magnitudes, their records, and the values these stand for."""
    x = rand((S, N, D), seed) * torch.linspace(0.25, 4.0, S, device="cuda").bfloat16().view(S, 1, 1)
    rows = attnres_cache_write(x, bits=bits, key_rank=R, key_offset=ko)
    return x, rows, attnres_cache_load(rows, D, bits=bits)


# ------------------------------------------------------------- write and load
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,R,ko", [(8, 8, 0), (8, 1, 7), (24, 5, 3), (40, 40, 0), (64, 33, 31), (200, 77, 100),
                                    (1000, 201, 733), (1024, 1024, 0), (4096, 1024, 2048), (8192, 8192, 0)])
def test_records_byte_for_byte(D, R, ko, bits):
    n = 5
    x = rand((n, D), D + bits)
    x[1] *= 1e-3
    x[2, : D // 2] = 0
    x[3, ::3] *= 300
    rows = attnres_cache_write(x, bits=bits, key_rank=R, key_offset=ko).cpu().numpy()
    codes, stat, size = ref.offsets(D, bits)
    assert rows.shape == (n, size) and attnres_cache_row_bytes(D, bits) == size
    back = np64(attnres_cache_load(torch.from_numpy(rows).cuda(), D, bits=bits))
    for i in range(n):
        rec, vals = ref.write_row(np64(x[i]), bits, R, ko)
        want = np.frombuffer(bytes(rec), np.uint8)
        off = np.abs(rows[i, stat:stat + 4].view(np.float32) - want[stat:stat + 4].view(np.float32))
        assert off <= 64 * ref.U * want[stat:stat + 4].view(np.float32)
        same = rows[i] == want
        same[stat:stat + 4] = True
        assert same.all(), np.argwhere(~same)[:4]
        assert np.array_equal(back[i], vals)


@pytest.mark.parametrize("bits", [8, 4])
def test_every_bf16_value_and_tie(bits):
    # every bf16 number next to a group maximum that makes the scale 1, and every one as its group's maximum
    top = {8: 448.0, 4: 6.0}[bits]
    allv = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    allv = allv[torch.isfinite(allv.float())]
    small = allv[allv.float().abs() <= top]
    x = torch.zeros((small.numel() + 30) // 31 * 31, dtype=torch.bfloat16)
    x[:small.numel()] = small
    x = torch.cat([torch.full((x.numel() // 31, 1), top, dtype=torch.bfloat16), x.view(-1, 31)], 1)
    y = torch.zeros(allv.numel(), 32, dtype=torch.bfloat16)
    y[:, 5] = allv
    y[:, 7] = allv / 3
    for m in (x, y):
        got = np64(attnres_cache_load(attnres_cache_write(m.cuda(), bits=bits), 32, bits=bits))
        want = np.stack([ref.write_row(r, bits, 32, 0)[1] for r in m.double().numpy()])
        assert np.array_equal(got, want)


@pytest.mark.parametrize("bits", [8, 4])
def test_groups_with_nan_or_infinity_read_as_nan(bits):
    x = rand((3, 96), 1)
    x[0, 40] = float("nan")
    x[1, 95] = float("inf")
    x[2, 0] = -float("inf")
    back = attnres_cache_load(attnres_cache_write(x, bits=bits), 96, bits=bits)
    nan = torch.isnan(back).cpu()
    want = torch.zeros((3, 96), dtype=torch.bool)
    want[0, 32:64] = want[1, 64:] = want[2, :32] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("bits", [8, 4])
def test_strides_parts_and_neighbours(bits):
    D, N = 200, 37
    size = attnres_cache_row_bytes(D, bits)
    wide = rand((N, D + 56), 3)
    x = wide[:, 24:24 + D]                         # rows with a stride, starting 48 bytes in
    plain = attnres_cache_write(x.contiguous(), bits=bits)
    cache = torch.full((3, 64, size + 32), 0xA5, dtype=torch.uint8, device="cuda")
    out = cache[1, 9:9 + N, :size]
    attnres_cache_write(x, bits=bits, out=out)
    assert torch.equal(out, plain)
    rest = cache.clone()
    rest[1, 9:9 + N, :size] = 0xA5
    assert (rest == 0xA5).all()                    # nothing else was written
    dst = torch.full((N, D + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    attnres_cache_load(out, D, bits=bits, out=dst[:, 8:8 + D])
    assert torch.equal(dst[:, 8:8 + D], attnres_cache_load(plain, D, bits=bits))
    assert (dst[:, :8] == 7).all() and (dst[:, 8 + D:] == 7).all()
    odd = rand((N * D + 1,), 4)[1:].view(N, D)     # rows off the 16-byte boundary: copied, not refused
    assert torch.equal(attnres_cache_write(odd, bits=bits), attnres_cache_write(odd.clone(), bits=bits))


def test_no_tokens():
    x = torch.empty((2, 0, 64), dtype=torch.bfloat16, device="cuda")
    rows = attnres_cache_write(x, bits=4, key_rank=16)
    assert rows.shape == (2, 0, attnres_cache_row_bytes(64, 4))
    assert attnres_cache_load(rows, 64, bits=4).shape == (2, 0, 64)
    q, w = rand((16,), 1), rand((64,), 2)
    f = attnres_cached_fwd(rows, q, 64, bits=4, w_o=w)
    assert f["y"].shape == (0, 64) and f["alpha"].shape == (0, 2)
    g = attnres_cached_bwd(rows, q, f["y"], f, 64, bits=4, w_o=w)
    assert not g["dq_f32"].any() and not g["dw_o_f32"].any() and g["dvalues"].shape == (2, 0, 64)


# ------------------------------------------------------------- read, gradient
SHAPES = [
    # S, N, D, R, ko, live, norm, scale
    (1, 1, 8, 8, 0, False, False, 1.0),
    (2, 3, 8, 3, 4, True, True, 1.0),
    (3, 200, 40, 17, 20, False, True, 0.5),
    (4, 5, 64, 64, 0, True, False, 1.0),
    (5, 33, 72, 1, 71, False, False, 2.0),
    (9, 70, 136, 136, 0, True, True, 1.0),
    (7, 19, 264, 100, 100, False, True, -1.0),
    (13, 37, 520, 130, 390, True, True, 1.0),
    (6, 41, 1000, 201, 733, True, True, 1.0),
    (8, 2, 1024, 1024, 0, False, False, 1.0),
    (17, 9, 1032, 300, 732, False, True, 1.0),
    (10, 23, 2056, 520, 1001, True, False, 1.0),
    (3, 31, 1056, 1056, 0, True, True, 1.0),
    (10, 23, 2072, 700, 1300, True, True, 1.0),
    (5, 1300, 2048, 512, 1536, False, True, 1.0),
    (4, 450, 4096, 1024, 2048, False, True, 1.0),
    (11, 13, 5000, 5000, 0, True, True, 1.0),
    (40, 7, 6152, 3000, 3000, False, True, 1.0),
    (12, 11, 4104, 4104, 0, True, True, 1.0),
    (33, 6, 8192, 2048, 6144, True, True, 1.0),
    (127, 2, 512, 512, 0, True, True, 1.0),
    (128, 3, 8192, 8192, 0, False, True, 1.0),
    (128, 130, 8, 8, 0, False, True, 1.0),
]


@pytest.mark.parametrize("form", ["cta", "warp"])  # the read's two kernels; rows of up to 1024 channels have one
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("S,N,D,R,ko,live,norm,scale", SHAPES)
def test_read_and_gradient(S, N, D, R, ko, live, norm, scale, bits, form, monkeypatch):
    if form == "warp" and D <= 1024:
        pytest.skip("one kernel")
    monkeypatch.setenv("ATTNRES_CACHED_FWD", form)
    x, rows, v = sources(S, N, D, bits, R, ko, seed=S * 7 + D)
    lv = rand((N, D), 11) if live else None
    q = rand((R,), 12, R ** -0.5)
    w = (1 + 0.1 * rand((D,), 13)).bfloat16() if norm else None
    dy = rand((N, D), 14)
    how = dict(bits=bits, live=lv, w_o=w, scale=scale, key_offset=ko)
    f = attnres_cached_fwd(rows, q, D, **how)
    g = attnres_cached_bwd(rows, q, dy, f, D, **how)
    allv = v if lv is None else torch.cat([v, lv[None]])
    want = ref.read(np64(allv), np64(q), scale, ko, np64(w) if norm else None, np64(dy))
    for name in ("rstd", "logit", "alpha", "y") + (("o_rstd",) if norm else ()):
        ref.check(name, f[name], want[name])
    dv = g["dvalues"] if lv is None else torch.cat([g["dvalues"], g["d_live"][None]])
    ref.check("dvalues", dv, want["dvalues"])
    ref.check("dq_f32", g["dq_f32"], want["dq_f32"])
    assert torch.equal(g["dq"], g["dq_f32"].bfloat16())
    if norm:
        ref.check("dw_o_f32", g["dw_o_f32"], want["dw_o_f32"])
        assert torch.equal(g["dw_o"], g["dw_o_f32"].bfloat16())
    again, gain = attnres_cached_fwd(rows, q, D, **how), attnres_cached_bwd(rows, q, dy, f, D, **how)
    assert all(torch.equal(f[k], again[k]) for k in f if f[k] is not None)
    assert all(torch.equal(g[k], gain[k]) for k in g if g[k] is not None)


@pytest.mark.parametrize("bits", [8, 4])
def test_is_the_plain_read_of_the_values_read_back(bits):
    """The run of operators as used: each source written into its place of a cache, then read with the
    block schedule's partial sum, against the uncompressed operators on the values read back."""
    S, N, D, R = 9, 300, 1024, 256
    cache = [torch.empty((N, attnres_cache_row_bytes(D, bits)), dtype=torch.uint8, device="cuda") for _ in range(S)]
    for s in range(S):
        for a, b in ((0, 111), (111, N)):          # a prompt in two parts
            attnres_cache_write(rand((N, D), s)[a:b], bits=bits, key_rank=R, out=cache[s][a:b])
    v = [attnres_cache_load(c, D, bits=bits) for c in cache]
    partial, q, dy = rand((N, D), 50), rand((R,), 51, R ** -0.5), rand((N, D), 52)
    f = attnres_cached_fwd(cache, q, D, bits=bits, live=partial)
    g = attnres_cached_bwd(cache, q, dy, f, D, bits=bits, live=partial)
    pf = attnres_fwd(v + [partial], q)
    pg = attnres_bwd(v + [partial], q, dy, pf)
    want = ref.read(np64(torch.stack(v + [partial])), np64(q), 1.0, D - R, None, np64(dy))
    # both are within the bound of the definition, so within twice the bound of each other
    for name, a, b in [(n, f[n], pf[n]) for n in ("y", "alpha", "rstd", "logit")] + \
            [("dvalues", torch.stack(g["dvalues"] + [g["d_live"]]), torch.stack(pg["dvalues"])),
             ("dq_f32", g["dq_f32"], pg["dq_f32"])]:
        bound = 2 * want[name][1].reshape(a.shape)
        assert (np.abs(np64(a) - np64(b)) <= bound).all(), name


def test_packed_list_and_repeated_records():
    S, N, D, bits = 5, 21, 264, 8
    _, rows, _ = sources(S, N, D, bits, D, 0)
    q, dy = rand((D,), 1, D ** -0.5), rand((N, D), 2)
    f = attnres_cached_fwd(rows, q, D, bits=bits)
    fl = attnres_cached_fwd([r.clone() for r in rows], q, D, bits=bits)
    strided = torch.zeros((S, N + 3, rows.shape[-1] + 16), dtype=torch.uint8, device="cuda")
    strided[:, 3:, :rows.shape[-1]] = rows
    fs = attnres_cached_fwd(strided[:, 3:, :rows.shape[-1]], q, D, bits=bits)
    for o in (fl, fs):
        assert torch.equal(f["y"], o["y"]) and torch.equal(f["alpha"], o["alpha"])
    twice = [rows[0], rows[1], rows[0]]            # the same records at two places
    ft = attnres_cached_fwd(twice, q, D, bits=bits)
    fc = attnres_cached_fwd([t.clone() for t in twice], q, D, bits=bits)
    assert torch.equal(ft["y"], fc["y"])
    gt = attnres_cached_bwd(twice, q, dy, ft, D, bits=bits)
    gc = attnres_cached_bwd([t.clone() for t in twice], q, dy, fc, D, bits=bits)
    assert all(torch.equal(a, b) for a, b in zip(gt["dvalues"], gc["dvalues"])) and torch.equal(gt["dq"], gc["dq"])
    lead = attnres_cached_fwd(rows.view(S, 3, 7, -1), q, D, bits=bits)
    assert lead["y"].shape == (3, 7, D) and torch.equal(lead["y"].view(N, D), f["y"])
    one = attnres_cached_fwd(rows[:, 4], q, D, bits=bits)
    assert one["y"].shape == (D,) and torch.equal(one["y"], f["y"][4])


@pytest.mark.parametrize("bits", [8, 4])
def test_zero_rows_and_dominant_sources(bits):
    N, D = 6, 200
    x = rand((4, N, D), 5)
    x[:, 0] = 0                                    # every source zero: uniform weights, zero output
    x[1, 1] = 0
    rows = attnres_cache_write(x, bits=bits)
    v = attnres_cache_load(rows, D, bits=bits)
    q, w = rand((D,), 6, 4.0), rand((D,), 7)       # logits of tens: some weights vanish
    dy = rand((N, D), 8)
    f = attnres_cached_fwd(rows, q, D, bits=bits, w_o=w)
    g = attnres_cached_bwd(rows, q, dy, f, D, bits=bits, w_o=w)
    assert (f["alpha"][0] == 0.25).all() and not f["y"][0].any()
    want = ref.read(np64(v), np64(q), 1.0, 0, np64(w), np64(dy))
    for name in ("rstd", "logit", "alpha", "y", "o_rstd"):
        ref.check(name, f[name], want[name])
    for name in ("dvalues", "dq_f32", "dw_o_f32"):
        ref.check(name, g[name], want[name])


@pytest.mark.parametrize("qs", [2.0 ** -120, 2.0 ** -60, 1.0, 2.0 ** 60])
def test_queries_of_every_magnitude(qs):
    """Channels of the query far apart: the read keeps those that count."""
    S, N, D, bits = 3, 8, 96, 8
    _, rows, v = sources(S, N, D, bits, D, 0)
    q = rand((D,), 3, D ** -0.5)
    q[::5] *= 2.0 ** -12
    q[1::7] *= 2.0 ** -25
    q = (q.float() * qs).bfloat16()
    f = attnres_cached_fwd(rows, q, D, bits=bits, scale=min(1.0, 1.0 / qs))
    want = ref.read(np64(v), np64(q), min(1.0, 1.0 / qs), 0)
    for name in ("rstd", "logit", "alpha", "y"):
        ref.check(name, f[name], want[name])


def test_nan_outside_the_key_reaches_the_output_only():
    N, D = 4, 128
    x = rand((3, N, D), 5)
    x[1, 2, 100] = float("nan")                    # group 96..127; the key is 0..31
    rows = attnres_cache_write(x, bits=4, key_rank=32, key_offset=0)
    f = attnres_cached_fwd(rows, rand((32,), 6), D, bits=4, key_offset=0)
    assert torch.isfinite(f["alpha"]).all() and torch.isfinite(f["logit"]).all()
    nan = torch.isnan(f["y"]).cpu()
    want = torch.zeros((N, D), dtype=torch.bool)
    want[2, 96:] = True
    assert torch.equal(nan, want)
    x[1, 2, 3] = float("inf")                      # now in the key: the token has no weights
    rows = attnres_cache_write(x, bits=4, key_rank=32, key_offset=0)
    f = attnres_cached_fwd(rows, rand((32,), 6), D, bits=4, key_offset=0)
    assert torch.isnan(f["y"][2]).all() and torch.isnan(f["alpha"][2]).all() and torch.isfinite(f["y"][:2]).all()


def test_records_of_another_key_or_format_are_reported():
    D, N = 256, 6
    x = rand((2, N, D), 1)
    rows = attnres_cache_write(x, bits=8, key_rank=64)
    q = rand((64,), 2)
    attnres_cached_fwd(rows, q, D, bits=8)
    attnres_check_device_error()
    f = attnres_cached_fwd(rows, q, D, bits=8, key_offset=0)     # written for the last 64 channels
    with pytest.raises(AttnresError):
        attnres_check_device_error()
    assert torch.isnan(f["y"]).all()
    rows[1, 3] = 0                                               # never written
    f = attnres_cached_fwd(rows, q, D, bits=8)
    with pytest.raises(AttnresError):
        attnres_check_device_error()
    assert torch.isnan(f["y"][3]).all() and torch.isfinite(f["y"][:3]).all()
    assert torch.isnan(attnres_cache_load(rows[1, 3], D, bits=8)).all()
    with pytest.raises(AttnresError):
        attnres_check_device_error()
    attnres_check_device_error()


# ------------------------------------------------------- outputs, streams, graphs
@pytest.mark.parametrize("bits", [8, 4])
def test_stores_stay_inside(bits):
    """Gradient rows and the workspace between sentinel bytes."""
    S, N, D, R = 3, 45, 1000, 300
    _, rows, _ = sources(S, N, D, bits, R, 13)
    q, w, dy, lv = rand((R,), 1, R ** -0.5), rand((D,), 2), rand((N, D), 3), rand((N, D), 4)
    how = dict(bits=bits, live=lv, w_o=w, key_offset=13)
    f = attnres_cached_fwd(rows, q, D, **how)
    plain = attnres_cached_bwd(rows, q, dy, f, D, **how)
    buf = torch.full((S, N + 4, D + 64), -7.0, dtype=torch.bfloat16, device="cuda")
    dv = [buf[s, 2:2 + N, 32:32 + D] for s in range(S)]
    ws = torch.full((1 << 22,), 0xA5, dtype=torch.uint8, device="cuda")
    attnres_cached_bwd(rows, q, dy, f, D, dvalues=dv, workspace=ws[4096:-4096], **how)
    for s in range(S):
        assert torch.equal(dv[s], plain["dvalues"][s])
        dv[s].fill_(-7.0)
    assert (buf == -7).all() and (ws[:4096] == 0xA5).all() and (ws[-4096:] == 0xA5).all()
    part = attnres_cached_bwd(rows, q, dy, f, D, need_dvalues=False, need_dlive=False, **how)
    assert part["dvalues"] is None and part["d_live"] is None
    assert torch.equal(part["dq_f32"], plain["dq_f32"]) and torch.equal(part["dw_o_f32"], plain["dw_o_f32"])


def test_other_stream_and_graph():
    S, N, D, bits = 6, 64, 520, 4
    x, rows, _ = sources(S, N, D, bits, D, 0)
    q, w, dy = rand((D,), 1, D ** -0.5), rand((D,), 2), rand((N, D), 3)

    def step():
        r = attnres_cache_write(x, bits=bits)
        f = attnres_cached_fwd(r, q, D, bits=bits, w_o=w)
        return attnres_cache_load(r, D, bits=bits), f, attnres_cached_bwd(r, q, dy, f, D, bits=bits, w_o=w)

    v, f, g = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        v2, f2, g2 = step()
    side.synchronize()
    graphs = []
    for _ in range(2):                             # two graphs, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    x.copy_(rand((S, N, D), 77))
    v3, f3, g3 = step()
    for graph, _ in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    for want, got in [((v, f, g), (v2, f2, g2))] + [((v3, f3, g3), out) for _, out in graphs]:
        assert torch.equal(want[0], got[0])
        for a, b in ((want[1], got[1]), (want[2], got[2])):
            assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)


@pytest.mark.parametrize("raw", [False, True])
def test_stream_argument(raw):
    """A call on `stream` waits for nothing on the current one: the copies of
    inputs that cannot be addressed in place, and what it allocates, are the
    stream's too."""
    S, N, D, bits = 3, 33, 136, 8
    x, rows, _ = sources(S, N, D, bits, D, 0)
    q, w, dy = rand((D,), 1, D ** -0.5), rand((D,), 2), rand((N, D), 3)
    f = attnres_cached_fwd(rows, q, D, bits=bits, w_o=w)
    g = attnres_cached_bwd(rows, q, dy, f, D, bits=bits, w_o=w)
    odd = torch.empty(rows.numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(rows.shape)
    odd.copy_(rows)
    xt, dyt, wide = x.transpose(1, 2).contiguous().transpose(1, 2), dy.t().contiguous().t(), rand((2 * D,), 5)
    w2 = wide[::2].copy_(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                  # some 50 ms on the current stream
    s = dict(bits=bits, stream=side.cuda_stream if raw else side)
    r2 = attnres_cache_write(xt, **s)
    v2 = attnres_cache_load(odd, D, **s)
    f2 = attnres_cached_fwd(odd, q, D, w_o=w2, **s)
    g2 = attnres_cached_bwd(odd, q, dyt, f2, D, w_o=w2, **s)
    side.synchronize()
    got = [t.cpu() for t in (r2, v2, f2["y"], f2["alpha"], g2["dvalues"], g2["dq_f32"], g2["dw_o_f32"])]
    want = [rows, attnres_cache_load(rows, D, bits=bits), f["y"], f["alpha"], g["dvalues"], g["dq_f32"], g["dw_o_f32"]]
    for a, b in zip(got, want):
        assert torch.equal(a, b.cpu())
    with pytest.raises(ValueError):
        attnres_cached_fwd([], q, D, **s)


# ----------------------------------------------------------------- autograd
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("bits", [8, 4])
def test_autograd(bits, packed):
    S, N, D, R = 4, 30, 264, 64
    x, rows, v = sources(S, N, D, bits, R, D - R)
    rows = rows if packed else [r.clone() for r in rows]
    vals = x.clone().requires_grad_() if packed else [t.clone().requires_grad_() for t in x]
    lv, q, w = rand((N, D), 1).requires_grad_(), rand((R,), 2, R ** -0.5).requires_grad_(), rand((D,), 3).requires_grad_()
    dy = rand((N, D), 4)
    y = attnres_cached(rows, q, D, bits=bits, values=vals, live=lv, out_norm_weight=w)
    leaves = [vals] if packed else list(vals)
    got = torch.autograd.grad(y, leaves + [lv, q, w], dy)
    f = attnres_cached_fwd(rows, q.detach(), D, bits=bits, live=lv.detach(), w_o=w.detach())
    g = attnres_cached_bwd(rows, q.detach(), dy, f, D, bits=bits, live=lv.detach(), w_o=w.detach())
    want = ([g["dvalues"]] if packed else list(g["dvalues"])) + [g["d_live"], g["dq"], g["dw_o"]]
    assert torch.equal(y, f["y"]) and all(torch.equal(a, b) for a, b in zip(got, want))
    # without values: the records are constants
    y2 = attnres_cached(rows, q, D, bits=bits, live=lv, out_norm_weight=w)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y2, [lv, q, w], dy), want[-3:]))


def test_overwritten_records_are_noticed_before_the_backward():
    S, N, D = 3, 10, 64
    rows = [attnres_cache_write(rand((N, D), s), bits=8) for s in range(S)]
    later = torch.empty_like(rows[0])
    q = rand((D,), 9).requires_grad_()
    y = attnres_cached(rows, q, D)
    attnres_cache_write(rand((N, D), 20), bits=8, out=later)     # another source: allowed
    torch.autograd.grad(y, q, torch.ones_like(y), retain_graph=True)
    attnres_cache_write(rand((N, D), 21), bits=8, out=rows[1])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, q, torch.ones_like(y))


def test_compiles_whole():
    S, N, D, bits = 3, 40, 128, 4
    x = rand((S, N, D), 1)
    q = rand((D,), 2, D ** -0.5).requires_grad_()

    def step(x, q):
        rows = attnres_cache_write(x, bits=bits)
        return attnres_cached(rows, q, D, bits=bits), attnres_cache_load(rows, D, bits=bits)

    y, v = step(x, q)
    cy, cv = torch.compile(step, fullgraph=True, backend="aot_eager")(x, q)
    assert torch.equal(y, cy) and torch.equal(v, cv)
    dy = rand((N, D), 3)
    assert torch.equal(torch.autograd.grad(y, q, dy)[0], torch.autograd.grad(cy, q, dy)[0])


@pytest.mark.parametrize("bits", [8, 4])
def test_gradient_against_differences(bits):
    """The gradient of sum(y * dy) in the query, the weight and the live source against central differences
    of the 64-bit definition, which the other tests hold the kernels to."""
    S, N, D, R, ko = 3, 4, 72, 30, 20
    _, rows, v = sources(S, N, D, bits, R, ko)
    lv, q, w, dy = rand((N, D), 1), rand((R,), 2, R ** -0.5), rand((D,), 3), rand((N, D), 4)
    how = dict(bits=bits, live=lv, w_o=w, key_offset=ko)
    f = attnres_cached_fwd(rows, q, D, **how)
    g = attnres_cached_bwd(rows, q, dy, f, D, **how)
    allv, q64, w64, dy64 = np64(torch.cat([v, lv[None]])), np64(q), np64(w), np64(dy)

    def loss(allv, q, w):
        return (ref.read(allv, q, 1.0, ko, w)["y"][0] * dy64).sum()

    want = ref.read(allv, q64, 1.0, ko, w64, dy64)
    rng, h = np.random.RandomState(0), 2.0 ** -14
    for got, arr, bound, call in [
            (np64(g["dq_f32"]), q64, want["dq_f32"][1], lambda a: loss(allv, a, w64)),
            (np64(g["dw_o_f32"]), w64, want["dw_o_f32"][1], lambda a: loss(allv, q64, a)),
            (np64(torch.cat([g["dvalues"], g["d_live"][None]])), allv, want["dvalues"][1], lambda a: loss(a, q64, w64))]:
        for _ in range(12):
            i = tuple(rng.randint(n) for n in arr.shape)
            up, down = arr.copy(), arr.copy()
            up[i] += h
            down[i] -= h
            slope = (call(up) - call(down)) / (2 * h)
            # h^2 / 6 times a third derivative; these are of order 10 for inputs of order 1
            assert abs(got[i] - slope) <= bound[i] + 20 * h * h + 1e-9


def test_inference_mode():
    """Serving: a cache made and filled under inference mode, and read from outside it."""
    with torch.inference_mode():
        cache = torch.empty((2, 4, attnres_cache_row_bytes(64, 4)), dtype=torch.uint8, device="cuda")
        for s in range(2):
            attnres_cache_write(rand((4, 64), s), bits=4, out=cache[s])
        q = rand((64,), 5)
        a = attnres_cached(cache, q, 64, bits=4)
        b = attnres_cached_fwd(cache, q, 64, bits=4)["y"]
    attnres_cache_write(rand((4, 64), 1), bits=4, out=cache[1])
    c = attnres_cached_fwd(cache, q, 64, bits=4)["y"]
    assert torch.equal(a, b) and torch.equal(b, c)


@pytest.mark.parametrize("form", ["cta", "warp"])
@pytest.mark.parametrize("bits,D", [(8, 200), (4, 200), (8, 2072), (4, 4096)])
def test_forward_stores_stay_inside(bits, D, form, monkeypatch):
    """Every output of the read between sentinel values, written whole; rows of a longer buffer behind the last
    token stay as they are."""
    monkeypatch.setenv("ATTNRES_CACHED_FWD", form)
    S, N = 3, 21
    _, rows, _ = sources(S, N, D, bits, D, 0)
    q, w, lv = rand((D,), 1, D ** -0.5), rand((D,), 2), rand((N, D), 3)
    how = dict(bits=bits, live=lv, w_o=w)
    plain = attnres_cached_fwd(rows, q, D, **how)
    bufs = {k: torch.full((N + 6,) + v.shape[1:], -7.0, dtype=v.dtype, device="cuda") for k, v in plain.items()}
    got = attnres_cached_fwd(rows, q, D, out={k: v[2:2 + N] for k, v in bufs.items()}, **how)
    for k, v in plain.items():
        assert torch.equal(got[k], v) and got[k].data_ptr() == bufs[k][2:].data_ptr()
        assert (bufs[k][:2] == -7).all() and (bufs[k][2 + N:] == -7).all(), k


@pytest.mark.parametrize("form", ["cta", "warp"])
def test_offsets_beyond_32_bits(form, monkeypatch):
    """A source of more than 4 GB of records: the last tokens are read, and their gradients written, like any."""
    monkeypatch.setenv("ATTNRES_CACHED_FWD", form)   # the same sums in the same order, whatever the length
    D, N, bits, tail = 4096, 1_100_000, 8, 5
    size = attnres_cache_row_bytes(D, bits)
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB")
    first, last = rand((1, D), 1), rand((tail, D), 2)
    rows = torch.empty((1, N, size), dtype=torch.uint8, device="cuda")
    assert rows.numel() > 1 << 32
    rows[0] = attnres_cache_write(first, bits=bits)
    attnres_cache_write(last, bits=bits, out=rows[0, N - tail:])
    q = rand((D,), 3, D ** -0.5)
    f = attnres_cached_fwd(rows, q, D, bits=bits)
    small = attnres_cached_fwd(rows[:, N - tail:].clone(), q, D, bits=bits)
    assert torch.equal(f["y"][N - tail:], small["y"]) and torch.equal(f["logit"][N - tail:], small["logit"])
    assert torch.equal(f["y"][:2], attnres_cache_load(rows[0, :2], D, bits=bits))     # one source: its values
    dy = f["y"]
    g = attnres_cached_bwd(rows, q, dy, f, D, bits=bits)
    gs = attnres_cached_bwd(rows[:, N - tail:].clone(), q, small["y"], small, D, bits=bits)
    assert torch.equal(g["dvalues"][:, N - tail:], gs["dvalues"])
    del g
    back = attnres_cache_load(rows[0], D, bits=bits)
    assert torch.equal(back[N - tail:], attnres_cache_load(attnres_cache_write(last, bits=bits), D, bits=bits))
    again = attnres_cache_write(back, bits=bits)[N - tail:]      # what codes stand for is kept exactly when written again
    assert torch.equal(attnres_cache_load(again, D, bits=bits), back[N - tail:])
