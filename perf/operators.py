"""The compressed source cache: what is measured of it, and its plain forms.

Every residual source of an Attention Residuals stack (the embedding, the
layers' or blocks' outputs) is written once and read by every later layer.
The cache holds a source's rows in 8 or 4 bits: per token one row record

    codes    D channels, 8 bits: one e4m3 byte a channel; 4 bits: one e2m1
             nibble a channel, channel 2i in the low half of byte i; padded
             with zeros to a multiple of 16 bytes
    scales   one byte per 32 channels: the exponent k of the group's scale 2^k,
             plus 127; padded to a multiple of 8 bytes
    stat     float32: the mean square of the row's key channels
             [key_offset, key_offset + R) as the codes stand for them
    tag      uint32: R | key_offset << 14 | (bits == 8) << 27 | 5 << 28
    pad      to a multiple of 16 bytes

k is the smallest exponent (-110 at least) for which the group's largest
magnitude is at most the type's (448 and 6) times 2^k, so nothing saturates;
codes are rounded to nearest, ties to even.  Dividing by 2^k is exact, and so
is reading a value back as bf16.

Four operators: write (quantise rows), load (read rows back), the softmax read
over cached rows (with an optional bf16 source that is not cached, read last),
and its gradient, which takes the cached values as the sources (dvalues is the
gradient of the values that the codes stand for).
"""
import math

import torch

own = False

GROUP = 32
EPS = 2.0 ** -23
LARGEST = {8: 448.0, 4: 6.0}
CLIP = 1.5 * 2.0 ** 127   # magnitudes above it are held as it: rounded up they would leave float32


# --------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a few sequences: the newest block sums go into the cache and come back; latency counts
        dict(name="round trip 8 bits, 4 tokens", op="trip", bits=8, N=4, D=4096, R=4096, ko=0),
        # a prefill's source at the long benchmark's width
        dict(name="round trip 4 bits, long", op="trip", bits=4, N=32768, D=4096, R=4096, ko=0),
        # odd token count and width, a key slice that starts and ends inside groups
        dict(name="round trip 8 bits, odd", op="trip", bits=8, N=5003, D=2056, R=520, ko=1001),
        # a pipeline stage gets nine cached sources and reads them back for a multi-query read
        dict(name="load 4 bits, nine sources", op="load", bits=4, S=9, N=8192, D=4096, R=1024, ko=512),
        # the smallest read: the quickstart's eight sources of two tokens
        dict(name="read 4 bits, two tokens", op="read", bits=4, S=8, N=2, D=1024, R=1024, ko=0, live=False, norm=False, scale=1.0),
        # the long workload (10 sources of 32768 tokens, output norm) from each type of cache
        dict(name="read 4 bits, long", op="read", bits=4, S=10, N=32768, D=4096, R=4096, ko=0, live=False, norm=True, scale=1.0),
        dict(name="read 8 bits, long", op="read", bits=8, S=10, N=32768, D=4096, R=4096, ko=0, live=False, norm=True, scale=1.0),
        # the deep workload: 64 sources of the widest rows
        dict(name="read 4 bits, deep", op="read", bits=4, S=64, N=8192, D=8192, R=8192, ko=0, live=False, norm=True, scale=1.0),
        # the block schedule: eight cached block sums and the current partial sum, quarter-rank keys
        dict(name="read 8 bits, block", op="read", bits=8, S=9, N=16384, D=4096, R=1024, ko=0, live=True, norm=False, scale=1.0),
        # training steps (the read and its gradient): the long workload, the block schedule, odd sizes
        dict(name="step 8 bits, long", op="step", bits=8, S=10, N=32768, D=4096, R=4096, ko=0, live=False, norm=True, scale=1.0),
        dict(name="step 4 bits, block", op="step", bits=4, S=9, N=16384, D=4096, R=1024, ko=2048, live=True, norm=False, scale=1.0),
        dict(name="step 8 bits, odd", op="step", bits=8, S=5, N=1003, D=1000, R=201, ko=733, live=True, norm=True, scale=0.5),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["trip", "load", "read", "read", "step"])
    D = 8 * _spread(rng, 8, 1024)
    R = D if rng.random() < 0.4 else rng.randint(1, D)
    ko = 0 if R == D else rng.choice([0, D - R, rng.randint(0, D - R)])
    case = dict(op=op, bits=rng.choice([8, 4]))
    if op == "trip":
        case.update(N=_spread(rng, 1, 32768), D=D, R=R, ko=ko)
        return case
    S = _spread(rng, 1, 64)
    most = (1 << 30) // (S * D)
    case.update(S=S, N=_spread(rng, 1, max(2, min(32768, most))), D=D, R=R, ko=ko)
    if op != "load":
        case.update(live=S > 1 and rng.random() < 0.5, norm=rng.random() < 0.5, scale=rng.choice([1.0, 0.5]))
    return case


# ------------------------------------------------------------------- layout
def _up(n, m):
    return (n + m - 1) // m * m


def _sizes(D, bits):
    """Where a row's scales, statistic and tag begin, and its bytes."""
    codes = _up(D * bits // 8, 16)
    stat = codes + _up(_up(D, GROUP) // GROUP, 8)
    return codes, stat, stat + 4, _up(stat + 8, 16)


def _tag(R, ko, bits):
    return R | ko << 14 | (bits == 8) << 27 | 5 << 28


def _grouped(x):
    """[..., D] as float32 [..., groups, 32], zeros behind the last channel."""
    D = x.shape[-1]
    x = torch.nn.functional.pad(x.float(), (0, _up(D, GROUP) - D))
    return x.view(*x.shape[:-1], -1, GROUP)


def _write(x, bits, R, ko):
    """Row records of bf16 rows, from elementary operations."""
    D = x.shape[-1]
    codes_at, stat_at, tag_at, size = _sizes(D, bits)
    g = _grouped(x)
    finite = torch.isfinite(g).all(-1, keepdim=True)
    g = torch.where(finite, g, 0.0).clamp(-CLIP, CLIP)
    m, e = torch.frexp(g.abs().amax(-1, keepdim=True))
    if bits == 8:                                    # 448 = 0.875 * 2^9
        k = e - 9 + (m > 0.875)
    else:                                            # 6 = 0.75 * 2^3
        k = e - 3 + (m > 0.75)
    k = k.clamp(min=-110)
    u = g * _two(-k)
    if bits == 8:
        codes = u.to(torch.float8_e4m3fn)
        back = codes.float() * _two(k)
        codes = codes.view(torch.uint8).flatten(-2)
    else:
        a = u.abs()                                  # magnitudes 0 0.5 1 1.5 2 3 4 6; a tie goes to the even code
        c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
        c = c | (torch.signbit(u).to(torch.uint8) << 3)
        back = _e2m1(c) * _two(k)
        c = c.flatten(-2)
        codes = c[..., 0::2] | c[..., 1::2] << 4
    back = torch.where(finite, back, math.nan).flatten(-2)
    stat = (back[..., ko:ko + R].square().sum(-1, dtype=torch.float64) / R).float()
    rows = torch.zeros((*x.shape[:-1], size), dtype=torch.uint8, device=x.device)
    n = min(codes.shape[-1], codes_at)
    rows[..., :n] = codes[..., :n]
    rows[..., codes_at:codes_at + k.shape[-2]] = torch.where(finite, k + 127, 255).squeeze(-1).to(torch.uint8)
    rows[..., stat_at:stat_at + 4] = stat.unsqueeze(-1).contiguous().view(torch.uint8)
    rows[..., tag_at:tag_at + 4] = torch.full((1,), _tag(R, ko, bits), dtype=torch.int32, device=x.device).view(torch.uint8)
    return rows


def _two(k):
    """2^k in float32 for whole k from -126 to 127."""
    return (k.int() + 127 << 23).view(torch.float32)


def _e2m1(c):
    """The value of e2m1 codes (0 to 15)."""
    m = torch.arange(8, dtype=torch.int32, device=c.device)
    table = torch.where(m < 2, m * 0.5, (m & 1 | 2) * _two((m >> 1) - 2))   # 0 0.5, then 2 or 3 times 2^(exponent - 2)
    return torch.cat([table, -table])[c.int()]


def _read_back(rows, D, bits):
    """float32 [..., D]: the values that row records stand for."""
    codes_at = _sizes(D, bits)[0]
    if bits == 8:
        v = rows[..., :D].contiguous().view(torch.float8_e4m3fn).float()
    else:
        b = rows[..., :D // 2]
        v = _e2m1(torch.stack((b & 15, b >> 4), -1).flatten(-2))
    scale = _two(rows[..., codes_at:codes_at + _up(D, GROUP) // GROUP].int() - 127)
    return v * scale.repeat_interleave(GROUP, -1)[..., :D]


# -------------------------------------------------------------- plain forms
def _sources(state):
    """float32 [S, N, D]: the cached sources, then the live one."""
    c = state["case"]
    v = _read_back(state["rows"], c["D"], c["bits"])
    return v if state["live"] is None else torch.cat([v, state["live"].float()[None]])


def _read(c, v, q, w):
    key = slice(c["ko"], c["ko"] + c["R"])
    t = v[..., key]
    rstd = torch.rsqrt(t.square().mean(-1) + EPS)                       # [S, N]
    logit = c["scale"] * rstd * torch.matmul(t, q)
    e = torch.exp(logit - logit.amax(0))
    alpha = e / e.sum(0)
    o = (alpha.unsqueeze(-1) * v).sum(0)
    o_rstd = torch.rsqrt(o.square().mean(-1) + EPS)
    y = o if w is None else o * o_rstd.unsqueeze(-1) * w
    return y, o, o_rstd, alpha, rstd, logit


def _plain_read(state):
    c = state["case"]
    q, w = state["q"].float(), None if state["w"] is None else state["w"].float()
    y, _, o_rstd, alpha, rstd, logit = _read(c, _sources(state), q, w)
    out = {"y": y.bfloat16(), "alpha": alpha.t().contiguous(), "rstd": rstd.t().contiguous(), "logit": logit.t().contiguous()}
    if w is not None:
        out["o_rstd"] = o_rstd
    return out


def _plain_step(state):
    c = state["case"]
    q, w = state["q"].float(), None if state["w"] is None else state["w"].float()
    v, dy = _sources(state), state["dy"].float()
    y, o, o_rstd, alpha, rstd, logit = _read(c, v, q, w)
    out = {"y": y.bfloat16()}
    do = dy
    if w is not None:
        r = o_rstd.unsqueeze(-1)
        out["dw_o_f32"] = (dy * o * r).sum(0)
        h = dy * w
        do = r * (h - o * r.square() * (h * o).mean(-1, keepdim=True))
    da = (do * v).sum(-1)
    dz = alpha * (da - (alpha * da).sum(0))                              # [S, N]
    key = slice(c["ko"], c["ko"] + c["R"])
    t = v[..., key]
    g = c["scale"] * dz * rstd
    out["dq_f32"] = torch.matmul(g.reshape(1, -1), t.reshape(-1, c["R"])).view(-1)
    dv = alpha.unsqueeze(-1) * do
    dv[..., key] += g.unsqueeze(-1) * q - (dz * logit * rstd.square() / c["R"]).unsqueeze(-1) * t
    S = state["rows"].shape[0]
    out["dvalues"] = dv[:S].bfloat16()
    if state["live"] is not None:
        out["d_live"] = dv[S].bfloat16()
    return out


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "trip":
        rows = _write(state["x"], c["bits"], c["R"], c["ko"])
        at = _sizes(c["D"], c["bits"])[1]
        return {"values": _read_back(rows, c["D"], c["bits"]).bfloat16(), "mean_square": rows[..., at:at + 4].contiguous().view(torch.float32).view(-1)}
    if c["op"] == "load":
        return {"values": _read_back(state["rows"], c["D"], c["bits"]).bfloat16()}
    return _plain_read(state) if c["op"] == "read" else _plain_step(state)


def _own(state):
    import attention_residuals_gb300 as ar
    c = state["case"]
    D, bits = c["D"], c["bits"]
    if c["op"] == "trip":
        rows = ar.attnres_cache_write(state["x"], bits=bits, key_rank=c["R"], key_offset=c["ko"])
        at = _sizes(D, bits)[1]
        return {"values": ar.attnres_cache_load(rows, D, bits=bits), "mean_square": rows[..., at:at + 4].view(torch.float32).view(-1)}
    if c["op"] == "load":
        return {"values": ar.attnres_cache_load(state["rows"], D, bits=bits)}
    how = dict(bits=bits, live=state["live"], w_o=state["w"], eps=EPS, scale=c["scale"], key_offset=c["ko"])
    f = ar.attnres_cached_fwd(state["rows"], state["q"], D, **how)
    if c["op"] == "read":
        return {k: f[k] for k in ("y", "alpha", "rstd", "logit", "o_rstd") if f[k] is not None}
    g = ar.attnres_cached_bwd(state["rows"], state["q"], state["dy"], f, D, **how)
    return {"y": f["y"], **{k: g[k] for k in ("dw_o_f32", "dq_f32", "dvalues", "d_live") if g[k] is not None}}


# ------------------------------------------------------------------- inputs
def prepare(case, seed):
    """Sources N(0, 1) times one U[0.5, 2] scalar each, as the benchmark's; a
    query of length about 1; the output weight near 1; dy N(0, 1)."""
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def source():
        x = normal(c["N"], c["D"])
        return x.mul_(0.5 + 1.5 * torch.rand((), generator=gen, device="cuda")).bfloat16()

    if c["op"] == "trip":
        return {"case": c, "x": source()}
    S = c["S"] - bool(c.get("live"))
    rows = torch.empty((S, c["N"], _sizes(c["D"], c["bits"])[3]), dtype=torch.uint8, device="cuda")
    for s in range(S):
        rows[s] = _write(source(), c["bits"], c["R"], c["ko"])
    if c["op"] == "load":
        return {"case": c, "rows": rows}
    state = {"case": c, "rows": rows, "live": source() if c["live"] else None}
    state["q"] = (normal(c["R"]) * c["R"] ** -0.5).bfloat16()
    state["w"] = (1.0 + 0.1 * normal(c["D"])).bfloat16() if c["norm"] else None
    if c["op"] == "step":
        state["dy"] = normal(c["N"], c["D"]).bfloat16()
    return state


def work(case):
    """Bytes: rows without their padding, bf16 tensors and statistics, each
    once.  A step keeps the statistics and o to itself: it reads the rows, dy,
    q and w, and writes y, the gradients and the sums."""
    c = case
    N, D = c["N"], c["D"]
    row = D * c["bits"] // 8 + (D + GROUP - 1) // GROUP + 8
    if c["op"] == "trip":
        return {"bytes": N * (2 * 2 * D + 2 * row + 4), "flops": 6 * N * D}
    if c["op"] == "load":
        return {"bytes": c["S"] * N * (row + 2 * D), "flops": c["S"] * N * D}
    S = c["S"] - c["live"]
    read = S * row + c["live"] * 2 * D
    vectors = 2 * c["R"] + 2 * D * c["norm"]
    if c["op"] == "read":
        out = 2 * D + 12 * c["S"] + 4 * c["norm"]
        return {"bytes": N * (read + out) + vectors, "flops": N * c["S"] * (2 * c["R"] + 2 * D)}
    out = 2 * D + c["S"] * 2 * D
    return {"bytes": N * (read + 2 * D + out) + vectors + 4 * c["R"] + 4 * D * c["norm"], "flops": N * c["S"] * (8 * c["R"] + 6 * D)}


# -------------------------------------------------------- 64-bit definition
def _magnitudes(bits):
    """Every non-negative value of the type, in code order, in float64."""
    if bits == 4:
        return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    low = [i / 8 * 2.0 ** -6 for i in range(8)]
    return torch.tensor(low + [(1 + i / 8) * 2.0 ** (e - 7) for e in range(1, 16) for i in range(8)][:119], dtype=torch.float64, device="cuda")


def _power(k):
    """2^k in float64."""
    return ((k.long() + 1023) * 2 ** 52).view(torch.float64)


def _exact_trip(x, bits):
    """The nearest representable value of every channel, by search."""
    n, D = x.shape
    grid = _magnitudes(bits)
    wide = torch.zeros((n, -(-D // GROUP) * GROUP), dtype=torch.float64, device="cuda")
    wide[:, :D] = x.double()
    wide = wide.reshape(n, -1, GROUP)
    top = wide.abs().max(dim=2, keepdim=True).values.clamp(min=2.0 ** -140)
    k = torch.ceil(torch.log2(top / grid[-1]))
    k = torch.where(top > grid[-1] * _power(k), k + 1, k)            # log2 may be a hair off next to a power of two
    k = torch.where(top <= grid[-1] * _power(k - 1), k - 1, k).clamp(min=-110.0)
    a = (wide.abs() / _power(k)).contiguous()
    mid = (grid[1:] + grid[:-1]) / 2
    below, above = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    code = torch.where(below % 2 == 0, below, above)                     # they differ on a tie alone: the even one
    return (torch.sign(wide) * grid[code] * _power(k)).reshape(n, -1)[:, :D]


def _exact_rows(rows, D, bits):
    """The values of row records [n, bytes], from their bytes, in float64."""
    n = rows.shape[0]
    grid = _magnitudes(bits)
    if bits == 8:
        code = rows[:, :D].int()
        v = torch.where(code >= 128, -1.0, 1.0).double() * grid[(code & 127).clamp(max=126)]
    else:
        code = rows[:, :D // 2].int()
        code = torch.cat([(code % 16).unsqueeze(2), (code // 16).unsqueeze(2)], dim=2).reshape(n, D)
        v = torch.where(code >= 8, -1.0, 1.0).double() * grid[code % 8]
    at = -(-(D * bits // 8) // 16) * 16
    group = torch.arange(D, device="cuda") // GROUP
    return v * _power(rows[:, at + group].int() - 127)


def exact(case, seed):
    c, state = case, prepare(case, seed)
    N, D, bits = c["N"], c["D"], c["bits"]
    lo, hi = c["ko"], c["ko"] + c["R"]
    if c["op"] == "trip":
        parts = [_exact_trip(p, bits) for p in state["x"].split(4096)]
        return {"values": torch.cat(parts), "mean_square": torch.cat([(p[:, lo:hi] ** 2).sum(1) / c["R"] for p in parts])}
    rows = state["rows"]
    if c["op"] == "load":
        return {"values": torch.stack([torch.cat([_exact_rows(p, D, bits) for p in r.split(4096)]) for r in rows])}
    q = state["q"].double()
    w = state["w"].double() if c["norm"] else None
    S, Sc = c["S"], rows.shape[0]
    size = max(1, (1 << 27) // (S * D))
    out = {"y": [], "alpha": [], "rstd": [], "logit": [], "o_rstd": []}
    if c["op"] == "step":
        dq, dw = torch.zeros_like(q), torch.zeros(D, dtype=torch.float64, device="cuda")
        dvs = torch.empty((Sc, N, D), dtype=torch.float64, device="cuda")
        dlive = torch.empty((N, D), dtype=torch.float64, device="cuda")
    for a in range(0, N, size):
        b = min(N, a + size)
        vs = [_exact_rows(rows[s, a:b], D, bits) for s in range(Sc)]
        if c["live"]:
            vs.append(state["live"][a:b].double())
        rs = torch.stack([((v[:, lo:hi] ** 2).sum(1) / c["R"] + EPS) ** -0.5 for v in vs], 1)    # [n, S]
        zs = c["scale"] * rs * torch.stack([(v[:, lo:hi] * q).sum(1) for v in vs], 1)
        al = torch.softmax(zs, dim=1)
        o = sum(al[:, s:s + 1] * v for s, v in enumerate(vs))
        ro = ((o ** 2).sum(1, keepdim=True) / D + EPS) ** -0.5
        for name, x in (("y", o if w is None else o * ro * w), ("alpha", al), ("rstd", rs), ("logit", zs), ("o_rstd", ro[:, 0])):
            out[name].append(x)
        if c["op"] == "step":
            d = state["dy"][a:b].double()
            if w is not None:
                xhat = o * ro
                dw += (d * xhat).sum(0)
                d = d * w
                d = ro * (d - xhat * (d * xhat).sum(1, keepdim=True) / D)
            da = torch.stack([(d * v).sum(1) for v in vs], 1)
            dz = al * da - al * (al * da).sum(1, keepdim=True)
            for s, v in enumerate(vs):
                that = v[:, lo:hi] * rs[:, s:s + 1]                       # the normalised key; z = scale * <that, q>
                dthat = c["scale"] * dz[:, s:s + 1] * q
                dq += c["scale"] * (dz[:, s:s + 1] * that).sum(0)
                dv = al[:, s:s + 1] * d
                dv[:, lo:hi] += rs[:, s:s + 1] * (dthat - that * (dthat * that).sum(1, keepdim=True) / c["R"])
                (dvs[s] if s < Sc else dlive)[a:b] = dv
    out = {k: torch.cat(x) for k, x in out.items()}
    if w is None:
        del out["o_rstd"]
    if c["op"] == "read":
        return out
    got = {"y": out["y"], "dq_f32": dq}
    if w is not None:
        got["dw_o_f32"] = dw
    got["dvalues"] = dvs
    if c["live"]:
        got["d_live"] = dlive
    return got
