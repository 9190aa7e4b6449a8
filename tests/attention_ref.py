"""Plain float64 forms of the attention operators, for their tests, with the
size of the roundings each kernel makes (bounds the tests hold it to)."""
import math

import torch


def positions_of(lq, lk, dev):
    return torch.arange(lk - lq, lk, device=dev)


def attn(q, k, v, window, scale, do=None):
    """One sequence: q [Lq, Hq, d] at the last positions, k, v [Lk, Hk, d], all
    float64.  Returns a dict of o, lse (and dq, dk, dv), and of the weighted
    magnitudes the bounds are made of (a row without keys: o = 0, lse = -inf)."""
    (lq, Hq, d), (lk, Hk, _) = q.shape, k.shape
    G = Hq // Hk
    kk, vv = k.repeat_interleave(G, 1).transpose(0, 1), v.repeat_interleave(G, 1).transpose(0, 1)
    qq = q.transpose(0, 1)
    i, j = positions_of(lq, lk, q.device)[:, None], torch.arange(lk, device=q.device)[None]
    vis = j <= i
    if window:
        vis = vis & (j > i - window)
    s = qq @ kk.transpose(1, 2) * scale
    s = torch.where(vis, s, float("-inf"))
    lse = torch.logsumexp(s, -1) if lk else torch.full((Hq, lq), float("-inf"), dtype=torch.float64, device=q.device)
    p = torch.where(vis & (lse[..., None] > float("-inf")), torch.exp(s - lse[..., None]), 0.0)
    r = {"o": p @ vv, "lse": lse, "o_abs": p @ vv.abs(),
         "s_abs": (qq.abs() @ kk.abs().transpose(1, 2) * scale).amax().item() if lk and lq else 0.0}
    if do is not None:
        dd = do.transpose(0, 1)
        dp = dd @ vv.transpose(1, 2)
        delta = (dd * r["o"]).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        # what rounding the forward's o moves delta by, per unit of the rounding
        dd_abs = (dd.abs() * (r["o"].abs() + r["o_abs"])).sum(-1, keepdim=True)
        w = ds.abs() + p * dd_abs
        dp_abs = dd.abs() @ vv.abs().transpose(1, 2) + dd_abs
        fold = lambda x: x.reshape(Hk, G, lk, d).sum(1)
        r["dq"], r["dq_abs"], r["dq_mag"] = ds @ kk * scale, w @ kk.abs() * scale, (p * dp_abs) @ kk.abs() * scale
        r["dk"] = fold(ds.transpose(1, 2) @ qq * scale)
        r["dk_abs"] = fold(w.transpose(1, 2) @ qq.abs() * scale)
        r["dk_mag"] = fold((p * dp_abs).transpose(1, 2) @ qq.abs() * scale)
        r["dv"], r["dv_abs"] = fold(p.transpose(1, 2) @ dd), fold(p.transpose(1, 2) @ dd.abs())
        r["dv_mag"] = r["dv_abs"]
    return {n: x.transpose(0, 1) if torch.is_tensor(x) else x for n, x in r.items()}


def float32_part(lk, d, s_abs):
    """Relative error of a weight p (and of its sums) in float32: a score is a
    sum of d products and exp2's argument is rounded (both relative to the
    score's magnitude s_abs), the sums over lk keys add one rounding a term."""
    return 2.0 ** -24 * (2 * (d + 8) * (1.0 + s_abs) + 2 * lk + 64)


def step(dtype):
    """Half a step of the type, relative."""
    return torch.finfo(dtype).eps / 2


def check(got, ref, bound, label):
    got = got.double()
    bad = ~((got - ref).abs() <= bound)
    # equal infinities
    bad &= ~((got == ref) & torch.isinf(ref))
    worst = ((got - ref).abs() / bound.clamp(min=1e-300)).nan_to_num(0.0).amax().item() if got.numel() else 0.0
    print(f"{label}: {worst:.3f} of the bound", flush=True)
    assert not bad.any(), f"{label}: {int(bad.sum())} of {bad.numel()} values outside the bound"


def check_attn(got, ref, dtype, lk, d, label):
    """got: dict of o, lse (and dq, dk, dv) of one sequence.  Roundings to the
    tensor type: the output (half a step of the value), the weights as
    operands (half a step of each: half a step of the weighted magnitudes),
    in the backward also o inside delta."""
    h = step(dtype) if dtype != torch.float32 else 0.0
    f = float32_part(lk, d, ref["s_abs"])
    out = step(dtype)
    check(got["o"], ref["o"], out * ref["o"].abs() + (h * 1.01 + f) * ref["o_abs"] + 1e-37, label + " o")
    if got.get("lse") is not None:
        lse = ref["lse"]
        check(got["lse"], lse, f + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0), label + " lse")
    for n in ("dq", "dk", "dv"):
        if n in got:
            check(got[n], ref[n], out * ref[n].abs() + h * 1.02 * ref[n + "_abs"] + 4 * f * ref[n + "_mag"] + 1e-37,
                  f"{label} {n}")


def rope(x, w, freqs, pos, inter, norm, eps):
    """x [B, T, H, d] float64 -> float64"""
    y = x
    if norm:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * w
    if freqs is None:
        return y
    n = freqs.numel()
    ang = (pos.double()[..., None] * freqs)[:, :, None]
    c, s = torch.cos(ang), torch.sin(ang)
    a, b = (y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if inter else (y[..., :n], y[..., n:2 * n])
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((r, y[..., 2 * n:]), -1)


def quantise(x):
    """(values the e4m3 codes stand for, exponent bytes) of float64 rows x, by
    the definition."""
    amax = x.abs().amax(-1, keepdim=True)
    fin = torch.isfinite(x).all(-1, keepdim=True)
    a = torch.where(fin & (amax > 0), amax, 448.0)
    m, k = torch.frexp(a)
    e = torch.where(m <= 0.875, k - 9, k - 8).clamp(min=-126)
    # powers by exp2: torch.ldexp's pow is an ulp off for some on the GPU, which breaks ties
    y = x * torch.exp2(-e.double())
    mag = y.abs().clamp(min=2.0 ** -60)
    st = torch.exp2((torch.frexp(mag)[1].double() - 1).clamp(min=-6.0) - 3.0)
    y = torch.round(y / st) * st
    val = torch.where(fin, y * torch.exp2(e.double()), math.nan)
    byte = torch.where(fin, e + 127, 255)[..., 0]
    return val, byte.to(torch.uint8)
