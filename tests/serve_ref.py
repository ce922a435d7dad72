"""Plain 64-bit forms of the few-token operators, written from their definitions.

Everything here is elementary torch arithmetic in float64, on whatever device
the inputs are; nothing of the package is used.  `bound_*` are the errors that
the operators' roundings allow, derived where they stand.
"""
import torch

MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BF16 = 2.0 ** -8          # half a step of bf16, relative
FP32 = 2.0 ** -24


def decode(codes, scales, nan_from=255):
    """float64 values of codes [..., d/2], scales [..., d/32]; bytes from nan_from up are NaN."""
    mag = torch.tensor(MAG + tuple(-m for m in MAG), dtype=torch.float64, device=codes.device)
    v = mag[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    e8m0 = [2.0 ** (i - 127) if i < nan_from else float("nan") for i in range(256)]    # a table: exact powers
    s = torch.tensor(e8m0, dtype=torch.float64, device=codes.device)[scales.long()]
    return v * s.repeat_interleave(32, -1)


def sf_of(scales, fill=0xFF):
    """Scales [N, K/32] in the scale-factor layout; bytes of no scale hold `fill`."""
    N, nb = scales.shape
    ka = (nb + 3) // 4
    sf = torch.full(((N + 127) // 128 * ka * 512,), fill, dtype=torch.uint8, device=scales.device)
    r = torch.arange(N, device=scales.device)[:, None]
    j = torch.arange(nb, device=scales.device)[None]
    sf[(r // 128 * ka + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4] = scales
    return sf


def gemv(x, codes, scales):
    """(product, sum of |x b|, sum over chunks of 256 of max|x| times sum |b|) in float64."""
    b, xd = decode(codes, scales), x.double()
    bad = torch.isnan(b).any()
    y = xd @ b.T
    bb = torch.nan_to_num(b).abs() if bad else b.abs()
    pad = (0, -b.shape[1] % 256)
    xc = torch.nn.functional.pad(xd.abs(), pad).unflatten(-1, (-1, 256))
    bc = torch.nn.functional.pad(bb, pad).unflatten(-1, (-1, 256))
    return y, xd.abs() @ bb.T, xc.amax(-1) @ bc.sum(-1).T


def gemv_bound(y, ab, tail, K, bf16):
    """K exact products summed in fp32 in any order, each add off by at most
    2^-23 of the running sum of magnitudes (covers truncating adds), and the
    block scalings (exact, or off by 2^-23 of a block's sum near the ends of
    fp32: two more such units); an element of x below 2^-32 of the largest of
    its 256 channels is off by 2^-40 of that: the largest is 2^15 or more in
    fp16, whose subnormals have steps of 2^-24.  bf16 output: half a step of
    the value."""
    tol = (K + 2) * 2.0 ** -23 * ab + 2.0 ** -40 * tail
    return tol + BF16 * (y.abs() + tol) if bf16 else tol


def gather(codes, scales, table, n, num_pages, nan_from=255):
    """Positions 0 .. n-1 of one sequence as float64 [n, heads, d] and whether each is on a page."""
    page = codes.shape[2]
    pos = torch.arange(n, device=codes.device)
    j = pos // page
    p = torch.where(j < table.numel(), table[j.clamp(max=max(table.numel() - 1, 0))].long(), torch.full_like(j, -1)) \
        if table.numel() else torch.full_like(j, -1)
    on = (p >= 0) & (p < num_pages)
    q = p.clamp(0, max(num_pages - 1, 0))
    v = decode(codes[q, :, pos % page], scales[q, :, pos % page], nan_from)
    return torch.where(on[:, None, None], v, torch.zeros_like(v)), on


def attention(q, cache, table, cu, lens, scale, causal):
    """Output and its error bound, float64 [T, hq, d] (rows of no sequence NaN in both).

    Bound, row by row, with S = sum_j p_j |v_j| / l (the error scale of a
    weighted mean): a score is an fp32 sum of d exact products, scaled and
    reduced by the maximum in fp32, so it is off by at most
    e = scale * ((d + 2) * 2^-23 * max_j sum |q k| + 2^-40 * max|q| * max_j sum |k|) + 4 * 2^-24 * max_j |s|
    (q is brought to fp16 by a power of two: 2^-40 of its largest at most);
    each p_j is then off by the factor 1 + 2 e + 2^-21 (the exponential's own
    error), and half a bf16 step for the second product (2^-8); sums of up to
    L terms in fp32 add (L + 8) 2^-23; a numerator and a denominator; and
    half a bf16 step of the result.  Where the second product takes p in fp16,
    as p 2^15 times the position's scale relative to the largest, a term below
    fp16's normal numbers is off by half of its smallest step, 2^-25, times a
    code of at most 6: L 2^-40 * 6 * 2^(largest scale) in all, over a sum of
    probabilities that is at least 1 (the maximum's own).
    """
    kc, ks, vc, vs = cache
    T, hq, d = q.shape
    H = kc.shape[1]
    g = hq // H
    out = torch.full((T, hq, d), float("nan"), dtype=torch.float64, device=q.device)
    tol = out.clone()
    for b in range(len(lens)):
        lo, hi, n = cu[b], cu[b + 1], lens[b]
        if hi <= lo:
            continue
        n = max(n, 0)
        k, on = gather(kc, ks, table[b], n, kc.shape[0], 253)
        v, _ = gather(vc, vs, table[b], n, kc.shape[0], 253)
        for h in range(H):
            kk, vv = k[:, h], v[:, h]
            for j in range(h * g, h * g + g):
                qq = q[lo:hi, j].double()
                s = qq @ kk.T * scale
                pos = lens[b] - (hi - lo) + torch.arange(hi - lo, device=q.device)
                seen = on[None].expand(hi - lo, -1)
                if causal:
                    seen = seen & (torch.arange(n, device=q.device)[None] <= pos[:, None])
                anyseen = seen.any(-1)
                s = torch.where(seen, s, torch.full_like(s, -float("inf")))
                m = torch.where(anyseen[:, None], s, torch.zeros_like(s)).amax(-1, keepdim=True) if n else s.sum(-1, keepdim=True)
                p = torch.where(seen, torch.exp(s - m), torch.zeros_like(s))
                l = p.sum(-1, keepdim=True)
                # what a row does not see must not reach it: no 0 * NaN
                clean = torch.nan_to_num(vv)
                y = torch.where(anyseen[:, None], p @ clean / l, torch.zeros(hi - lo, d, dtype=torch.float64, device=q.device))
                hit = (seen.double() @ torch.isnan(vv).double()) > 0
                out[lo:hi, j] = torch.where(hit, torch.full_like(y, float("nan")), y)
                S = torch.nan_to_num(p) @ clean.abs() / torch.nan_to_num(l).clamp_min(1e-300)
                if n:
                    qk = torch.where(seen, qq.abs() @ torch.nan_to_num(kk).abs().T, torch.zeros_like(s)).amax(-1)
                    ka = torch.nan_to_num(kk).abs().sum(-1).amax()
                    top = torch.where(seen, s.abs(), torch.zeros_like(s)).nan_to_num().amax(-1)
                    e = abs(scale) * ((d + 2) * 2.0 ** -23 * qk + 2.0 ** -40 * qq.abs().amax(-1) * ka) + 4 * FP32 * top
                else:
                    e = torch.zeros(hi - lo, dtype=torch.float64, device=q.device)
                vtop = vs[table[b][(torch.arange(n, device=q.device) // kc.shape[2]).clamp(max=table.shape[1] - 1)].long().clamp(0, kc.shape[0] - 1), h,
                          torch.arange(n, device=q.device) % kc.shape[2]] if n and table.shape[1] else vs[:0, h, 0]
                vtop = torch.where((vtop < 253) & on[:, None], vtop, torch.zeros_like(vtop)).amax().item() if vtop.numel() else 0
                rel = 2 * (2 * e + 2.0 ** -21 + (n + 8) * 2.0 ** -23) + BF16
                tt = (rel[:, None] * S + n * 2.0 ** -40 * 6 * 2.0 ** (vtop - 127)) * (1 + BF16) + BF16 * y.abs()
                tol[lo:hi, j] = torch.where(hit, torch.zeros_like(tt), tt)
    return out, tol
