"""The 8-bit paged cache in 64 bits, from the definitions in include/nsa.h
(torch on the CPU, plain loops over sequences, pages and heads)."""
import math

import torch

F64 = torch.float64


def e4m3(x):
    """x (fp64, |x| <= 448 or NaN) rounded to e4m3's values, nearest, ties to even."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-6)
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e)  # log2 rounded up
    step = torch.exp2(e - 3)
    return (torch.round(a / step) * step).clamp(max=448.0) * torch.sign(x)  # NaN stays


def step_of(v):
    """Distance from e4m3 value magnitudes |v| to the next larger value."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 3)


def need(a):
    """Smallest power of two >= 2^-126 with a <= 448 * it."""
    s = 2.0 ** -126
    while a > 448.0 * s:
        s *= 2.0
    return s


def decode(pages):
    """float8 pages as fp64 values on the CPU."""
    return pages.detach().cpu().float().to(F64)


def turned(x, table, positions, style):
    """x [N, H, d] fp64 with row n rotated to positions[n] by table [len, 2, r / 2]."""
    t = table.detach().cpu().to(F64)[positions]
    c, s = t[:, 0, None], t[:, 1, None]
    half = t.shape[-1]
    y = x.clone()
    i = torch.arange(half)
    a, b = (i, i + half) if style == "half" else (2 * i, 2 * i + 1)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def tokens(cu, b):
    return (b, b + 1) if cu is None else (int(cu[b]), int(cu[b + 1]))


def attend(q, k_pages, v_pages, k_scale, v_scale, table, seq_lens, page, cu=None, keys="all",
           window=0, sel=None, scale=None):
    """(out, lse, A, B) in fp64: A [N, Hq, d] = sum p |v| / sum p and B [N, Hq] =
    the largest scale * sum |q_e k_e| over a row's keys, for error bounds. Rows
    outside the offsets are NaN."""
    q = q.detach().cpu().to(F64)
    N, Hq, d = q.shape
    Hkv = k_pages.shape[1]
    G = Hq // Hkv
    scale = scale or 1.0 / math.sqrt(d)
    kc, vc = decode(k_pages), decode(v_pages)
    ks, vs = k_scale.detach().cpu().to(F64), v_scale.detach().cpu().to(F64)
    table, lens = table.cpu(), seq_lens.cpu()
    out = torch.full_like(q, math.nan)
    lse = torch.full((N, Hq), math.nan, dtype=F64)
    A, Bz = torch.zeros_like(q), torch.zeros(N, Hq, dtype=F64)
    for b in range(table.shape[0]):
        lo, hi = tokens(cu, b)
        L, n = int(lens[b]), hi - lo
        for i in range(n):
            pos = L - n + i
            for g in range(Hkv):
                first = max(0, pos + 1 - window) if keys == "window" else 0
                want = list(range(first, pos + 1))
                if keys == "blocks":
                    blocks = {int(j) for j in sel[b, g] if j >= 0}
                    want = [x for x in want if x // page in blocks]
                row, hs = lo + i, slice(g * G, (g + 1) * G)
                if not want:
                    out[row, hs], lse[row, hs] = 0.0, -math.inf
                    continue
                x = torch.tensor(want)
                pid = table[b, x // page].long()
                live = (pid >= 0) & (pid < k_pages.shape[0])
                x, pid = x[live], pid[live]
                if not len(x):
                    out[row, hs], lse[row, hs] = 0.0, -math.inf
                    continue
                k = kc[pid, g, x % page] * ks[pid, g, None]
                v = vc[pid, g, x % page] * vs[pid, g, None]
                z = q[row, hs] @ k.T * scale
                top = z.amax(1, keepdim=True)
                p = torch.exp(z - top)
                total = p.sum(1, keepdim=True)
                out[row, hs] = p @ v / total
                lse[row, hs] = (top + total.log())[:, 0]
                A[row, hs] = p @ v.abs() / total
                Bz[row, hs] = (q[row, hs].abs() @ k.abs().T * abs(scale)).amax(1)
    return out, lse, A, Bz


def bounds(out, lse, A, B, dtype, keys_seen):
    """Largest errors of (out, lse) that the kernels' arithmetic allows.

    A score has at most 2^-22 relative from the query's parts and 48 additions
    (16 products a step, 8 steps, twice for fp32's two parts) of 2^-23 in fp32:
    dz <= B 2^-17. p has dz and 2^-21 from its exponentials. The weighted sum
    adds 2^-12 (fp16 p: half a step of 2^-11) for bf16 and 2^-22 for fp32's two
    parts, and one fp32 addition of 2^-23 for every 16 keys and every joined
    part; numerator and denominator both. The output is rounded once."""
    dz = B * 2.0 ** -17 + 2.0 ** -21
    adds = (keys_seen / 16 + 64) * 2.0 ** -23
    if dtype == torch.bfloat16:
        rel, final = 2.0 ** -11, 2.0 ** -8
    else:
        rel, final = 2.0 ** -21, 2.0 ** -24
    t_out = A * (2 * dz[..., None] + 2 * adds + rel) + final * out.abs() + 1e-30
    t_lse = dz + adds + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0) + 2.0 ** -22
    return t_out, t_lse


def append(k_new, v_new, pos, cu, pages, scales, table, page, rope=None, style="half"):
    """Definition of one append for K and V: a list of (name, expected codes,
    expected scales, x' rows, slack of x') with untouched places as they were."""
    table = table.cpu()
    got = []
    for name, x, pg, sc in (("k", k_new, pages[0], scales[0]), ("v", v_new, pages[1], scales[1])):
        x = x.detach().cpu().to(F64)
        slack = torch.zeros_like(x)
        B = table.shape[0]
        where = []
        for b in range(B):
            lo, hi = tokens(cu, b)
            where += [(r, b, int(pos[b]) + r - lo) for r in range(lo, hi)]
        if name == "k" and rope is not None and where:
            at = torch.tensor([w[2] for w in where])
            rows = torch.tensor([w[0] for w in where])
            both = torch.stack((x[rows].abs(), turned(x[rows].abs(), rope.abs(), at, style).abs()))
            slack[rows] = 2.0 ** -21 * both.amax(0).amax(-1, keepdim=True)
            x = x.clone()
            x[rows] = turned(x[rows], rope, at, style)
        codes, scale = decode(pg).clone(), sc.detach().cpu().to(F64).clone()
        groups = {}
        for r, b, t in where:
            groups.setdefault((b, t // page), []).append((r, t % page))
        for (b, j), rows in groups.items():
            pid = int(table[b, j])
            for h in range(x.shape[1]):
                vals = x[[r for r, _ in rows], h]
                fine = torch.isfinite(vals)
                a = float(vals[fine].abs().max()) if fine.any() else 0.0
                s = need(a)
                old = float(scale[pid, h])
                if rows[0][1] != 0:
                    s = max(old, s)
                if s != old:  # slots that the call does not write keep their values
                    other = codes[pid, h] * (old / s)
                    codes[pid, h] = torch.where(other.abs() > 464, math.nan, e4m3(other))
                scale[pid, h] = s
                for (r, slot), v, ok in zip(rows, vals, fine):
                    codes[pid, h, slot] = torch.where(ok, e4m3(torch.where(ok, v, 0.0) / s), math.nan)
        got.append((name, codes, scale, x, slack))
    return got
