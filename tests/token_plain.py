"""Plain 64-bit forms of the token loop's operators (for the tests): written
from the formulas in include/fastmamba.h, sharing nothing with the kernels."""
import torch

F64 = torch.float64


def blocks(n):
    return (n + 127) // 128


def e4m3_round(v):
    """v (fp64) to the nearest e4m3 value, ties to even, saturating at 448."""
    m, e = torch.frexp(v)  # |v| = m 2^e, m in [0.5, 1)
    unit = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return (torch.round(v / unit) * unit).clamp(-448.0, 448.0)


def norm(x, residual, w, eps, kind):
    """(r fp32, codes fp64, scales fp32, distance of each code's argument from a tie)"""
    r = x.float() if residual is None else x.float() + residual
    d = r.to(F64)
    M, K = d.shape
    y = d / torch.sqrt((d * d).sum(1, keepdim=True) / K + eps) * w.to(F64)
    width, top = (128, 448.0) if kind == "e4m3" else (K, 127.0)
    codes, scales, gap = torch.zeros_like(y), [], torch.ones_like(y)
    for b in range(-(-K // width)):
        at = slice(b * width, min(K, (b + 1) * width))
        a = y[:, at].abs().amax(1)
        a = torch.where(a >= 2.0 ** -100, a, 0.0)
        s = (a / top).float()
        v = torch.where(s[:, None] > 0, y[:, at] / s.to(F64)[:, None].clamp_min(2.0 ** -140), 0.0)
        codes[:, at] = e4m3_round(v) if kind == "e4m3" else torch.round(v).clamp(-127, 127)
        # relative distance to the next code's border
        near = codes[:, at]
        lo, hi = v * (1 - 2.0 ** -44), v * (1 + 2.0 ** -44)
        f = e4m3_round if kind == "e4m3" else (lambda t: torch.round(t).clamp(-127, 127))
        gap[:, at] = ((f(lo) == near) & (f(hi) == near)).to(F64)
        scales.append(s)
    return r, codes, torch.stack(scales, 1) if kind == "e4m3" else scales[0], gap


def dequant_rows(a, s):
    return a.to(torch.float32).to(F64) * s.to(F64).repeat_interleave(128, 1)[:, :a.shape[1]]


def dequant_blocks(w, s):
    return dequant_rows(w, s.repeat_interleave(128, 0)[:w.shape[0]])


def beam(logits, scores, finished, eos, n_out):
    """(scores fp64, parent, token, finished): every candidate of a beam in the
    order of its logits, the beams' lists merged by c."""
    B, k, V = logits.shape
    l = torch.nan_to_num(logits.to(F64), nan=-torch.inf, posinf=float(torch.finfo(torch.float32).max),
                         neginf=-torch.inf)
    order = torch.sort(l, dim=2, descending=True, stable=True).indices
    top = l.amax(2, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    lse = top + torch.log(torch.exp(l - top).sum(2, keepdim=True))
    sc = scores.to(F64)
    c = torch.where(l > -torch.inf, l - lse + sc[:, :, None], -torch.inf)
    lowest = torch.finfo(torch.float32).min
    out = torch.full((B, n_out), -torch.inf, dtype=F64)
    par = (torch.arange(n_out) % k).expand(B, n_out).clone()
    tok = torch.full((B, n_out), -1, dtype=torch.int64)
    nf = torch.zeros(B, n_out, dtype=torch.uint8)
    for b in range(B):
        lists = []
        for j in range(k):
            done = finished is not None and int(finished[b, j]) != 0
            if not float(sc[b, j]) > -torch.inf:
                lists.append([])
            elif done:
                lists.append([(float(sc[b, j]), eos, 1)])
            else:
                lists.append([(float(c[b, j, v]), int(v), int(int(v) == eos))
                              for v in order[b, j, :n_out] if float(c[b, j, v]) > -torch.inf])
        for n in range(n_out):
            j = max((j for j in range(k) if lists[j]), key=lambda j: (lists[j][0][0], -j), default=None)
            if j is None:
                break
            value, tok[b, n], nf[b, n] = lists[j].pop(0)
            out[b, n], par[b, n] = max(value, lowest), j
    return out, par, tok, nf
