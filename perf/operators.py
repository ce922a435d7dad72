"""The operators of a 4-bit transformer layer that answers a few tokens at a time, as cases to be measured.

  gemv       a few token rows times MXFP4 weights that are laid out for the W4A4 product (mxf4_gemv)
  cache      keys and values of new tokens quantized into a paged MXFP4 cache, and read back (mx_cache_write, mx_cache_read)
  read       positions of the cache back as bf16, whole sequences at a time (mx_cache_read)
  attention  attention of a chunk of new tokens over the paged MXFP4 cache (mx_paged_attention)

MXFP4: blocks of 32 channels, one E8M0 scale byte s (value 2^(s - 127)) and 32 E2M1 codes (sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte,
the even element in the low nibble. The cache has codes [pages, kv heads, page, head dim / 2] and scales [pages, kv heads, page, head dim / 32];
block_table [sequences, pages of the longest] names each sequence's pages; cu_seqlens [sequences + 1] says where each sequence's new tokens begin
among the rows; seq_lens [sequences] are the lengths with the new tokens, which are the last ones.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the modulation vectors of one sample from its time embedding (PixArt's width), the smallest product
        dict(name="gemv 1x1152x1152", op="gemv", m=1, n=1152, k=1152, f32=False),
        # SANA's widths, whose blocks fill no whole scale units and whose rows no whole group, an odd number of rows, fp32 out
        dict(name="gemv 5x5600x2240 f32", op="gemv", m=5, n=5600, k=2240, f32=True),
        # a decode step of a batch through a wide layer's down product: the largest weights
        dict(name="gemv 16x8192x28672", op="gemv", m=16, n=8192, k=28672, f32=False),
        # one new token for each of 64 sequences: a decode step's cache update
        dict(name="cache 64 tokens", op="cache", batch=64, past=900, new=1, hkv=8, d=128, page=64, f32=False),
        # a prompt of ragged sequences enters the cache, as fp32 from a transform
        dict(name="cache 16k tokens f32", op="cache", batch=5, past=0, new=4099, hkv=8, d=128, page=64, f32=True),
        # short sequences on small pages with narrow heads
        dict(name="read 3x700 d64", op="read", batch=3, past=700, new=0, hkv=4, d=64, page=16),
        # long sequences back as bf16, for another engine or a check
        dict(name="read 4x20000", op="read", batch=4, past=20000, new=0, hkv=8, d=128, page=64),
        # one sequence's next token, a short context: latency
        dict(name="decode 1x1000 d64", op="attention", batch=1, past=999, new=1, hq=16, hkv=4, d=64, page=16, causal=True),
        # a decode step of an ordinary batch of ragged sequences
        dict(name="decode 32x4096", op="attention", batch=32, past=4095, new=1, hq=32, hkv=8, d=128, page=64, causal=True),
        # a decode step over long contexts: the cache is the whole cost
        dict(name="decode 16x40000", op="attention", batch=16, past=40000, new=1, hq=64, hkv=8, d=128, page=64, causal=True),
        # chunks of two prompts over what is cached of them, ragged, an odd number of pages
        dict(name="chunk 2x777 of 3000", op="attention", batch=2, past=3000, new=777, hq=24, hkv=8, d=96, page=32, causal=True),
        # a large chunk of one long prompt: the products are the whole cost
        dict(name="chunk 2048 of 32000", op="attention", batch=1, past=30000, new=2048, hq=32, hkv=8, d=128, page=64, causal=True),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "cache", "read", "attention", "attention", "attention"])
    if op == "gemv":
        k = 32 * spread(rng, 4, 900)
        return dict(op=op, m=rng.randint(1, 32), n=spread(rng, 64, min(28672, 8192 * 28672 // k)), k=k, f32=rng.random() < 0.5)
    d = rng.choice([32, 64, 96, 128])
    page = rng.choice([16, 32, 48, 64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    batch = spread(rng, 1, 64)
    if op == "cache":
        return dict(op=op, batch=batch, past=rng.randint(0, 2000), new=spread(rng, 1, max(1, 16000 // batch)), hkv=hkv, d=d, page=page, f32=rng.random() < 0.5)
    if op == "read":
        return dict(op=op, batch=batch, past=spread(rng, 1, 80000 // batch), new=0, hkv=hkv, d=d, page=page)
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    if rng.random() < 0.5:
        return dict(op=op, batch=batch, past=spread(rng, 1, 300000 // batch), new=rng.choice([1, 1, 1, 2, 4, 5]), hq=hq, hkv=hkv, d=d, page=page, causal=rng.random() < 0.8)
    batch = rng.choice([1, 1, 2, 3, 5])
    new = spread(rng, 16, 2048 * 4096 // (max(4096, hq * d) * batch))
    return dict(op=op, batch=batch, past=spread(rng, 1, 30000 // batch), new=new, hq=hq, hkv=hkv, d=d, page=page, causal=rng.random() < 0.8)


def lengths(case):
    """Each sequence's cached and new tokens: the first has the case's numbers, the others are ragged, up to a third shorter."""
    rng = random.Random(case["batch"] * 1000003 + case["past"])
    less = lambda n: n - rng.randint(0, n // 3)  # noqa: E731
    past = [case["past"]] + [less(case["past"]) for _ in range(case["batch"] - 1)]
    new = [case["new"]] + [less(case["new"]) if case["new"] > 1 else case["new"] for _ in range(case["batch"] - 1)]
    return past, new


def quantized(x):
    """MXFP4 of the blocks x [..., 32]: codes 0..15 and scale bytes, by the OCP rule: 2^(floor(log2 amax) - 2), nearest code, ties to the even one."""
    amax = x.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    y = torch.ldexp(x, -e)
    a = y.abs()
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return code + 8 * torch.signbit(y), (e + 127)[..., 0]


def packed(code):
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)


def decoded(codes, scales):
    """fp32 values of codes [..., d / 2] and scales [..., d / 32]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    s = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def unit_offsets(rows, nb, device):
    """Where the scale of each (row, block) stands in the scale-factor layout."""
    r, j = torch.arange(rows, device=device)[:, None], torch.arange(nb, device=device)[None, :]
    return ((r // 128) * ((nb + 3) // 4) + j // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + j % 4


def fill(codes, scales, gain, gen):
    """A pool of pages with quantized normal values: rows of unlike sizes and a few loud channels, as keys and values have."""
    blocks = scales.numel()
    fc, fs = codes.view(blocks, 16), scales.view(blocks)
    d = codes.shape[-1] * 2
    loud = torch.exp(gain * torch.randn(d, device=codes.device, generator=gen)).view(-1, 32)
    for at in range(0, blocks, 1 << 22):
        n = min(1 << 22, blocks - at)
        x = torch.randn(n, 32, device=codes.device, generator=gen)
        x *= loud[(torch.arange(at, at + n, device=codes.device) % (d // 32))]
        c, s = quantized(x)
        fc[at:at + n], fs[at:at + n] = packed(c), s.to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = dict(case)
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"] = (torch.randn(m, k, device=dev, generator=gen) * torch.exp(0.5 * torch.randn(k, device=dev, generator=gen))).bfloat16()
        c, s = quantized(torch.randn(n, k // 32, 32, device=dev, generator=gen) / math.sqrt(k))
        st["codes"] = packed(c).view(n, k // 2)
        sf = torch.zeros((n + 127) // 128 * ((k // 32 + 3) // 4) * 512, dtype=torch.uint8, device=dev)
        sf[unit_offsets(n, k // 32, dev)] = s.to(torch.uint8)
        st["sf"] = sf
        return st
    past, new = lengths(case)
    lens = [p + n for p, n in zip(past, new)]
    page, hkv, d = case["page"], case["hkv"], case["d"]
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + 7  # a few pages of the pool belong to no sequence
    order = torch.randperm(pages, device=dev, generator=gen).int()
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st["table"] = table
    for t in "kv":
        st[t + "c"] = torch.empty(pages, hkv, page, d // 2, dtype=torch.uint8, device=dev)
        st[t + "s"] = torch.empty(pages, hkv, page, d // 32, dtype=torch.uint8, device=dev)
        fill(st[t + "c"], st[t + "s"], 0.6 if t == "k" else 0.2, gen)
    cum = lambda v: torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], dtype=torch.int32, device=dev)  # noqa: E731
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["starts"] = torch.tensor(past, dtype=torch.int32, device=dev)
    st["max_len"], st["max_new"] = max(lens), max(new)
    if case["op"] == "read":
        st["cu"], st["rows"] = cum(lens), sum(lens)
        return st
    st["cu"], st["rows"] = cum(new), sum(new)
    if case["op"] == "cache":
        # the keys and values of a fused projection's rows, token by token
        kv = torch.randn(st["rows"], 2 * hkv, d, device=dev, generator=gen) * torch.exp(0.4 * torch.randn(2 * hkv, d, device=dev, generator=gen))
        kv = kv if case["f32"] else kv.bfloat16()
        st["k"], st["v"] = kv[:, :hkv], kv[:, hkv:]
    else:
        st["q"] = torch.randn(st["rows"], case["hq"], d, device=dev, generator=gen).bfloat16()
    return st


def rows_of(st):
    """Sequence and position of every row."""
    row = torch.arange(st["rows"], device=st["cu"].device)
    seq = torch.searchsorted(st["cu"][1:].long(), row, right=True)
    return seq, row - st["cu"][seq]


def run(state):
    st = state
    if own:
        import w4a4_mxfp4_post_b200 as kq

        if st["op"] == "gemv":
            return kq.mxf4_gemv(st["x"], st["codes"], st["sf"], out_dtype=torch.float32 if st["f32"] else torch.bfloat16)
        if st["op"] == "read":
            return kq.mx_cache_read(st["kc"], st["ks"], st["vc"], st["vs"], st["table"], st["cu"], st["rows"])
        if st["op"] == "cache":
            kq.mx_cache_write(st["k"], st["v"], st["kc"], st["ks"], st["vc"], st["vs"], st["table"], st["cu"], st["lens"])
            return kq.mx_cache_read(st["kc"], st["ks"], st["vc"], st["vs"], st["table"], st["cu"], st["rows"], starts=st["starts"])
        return kq.mx_paged_attention(st["q"], st["kc"], st["ks"], st["vc"], st["vs"], st["table"], st["cu"], st["lens"], max_new=st["max_new"], causal=st["causal"])
    if st["op"] == "gemv":
        n, k = st["n"], st["k"]
        w = decoded(st["codes"], st["sf"][unit_offsets(n, k // 32, st["sf"].device)])
        y = st["x"].float() @ w.T
        return y if st["f32"] else y.bfloat16()
    if st["op"] in ("read", "cache"):
        seq, pos = rows_of(st)
        if st["op"] == "cache":
            pos = pos + st["starts"][seq]
        page = st["table"][seq, pos // st["page"]].long()
        at = pos % st["page"]
        if st["op"] == "cache":
            kc, ks = quantized(st["k"].float().unflatten(-1, (-1, 32)))
            vc, vs = quantized(st["v"].float().unflatten(-1, (-1, 32)))
            st["kc"][page, :, at], st["ks"][page, :, at] = packed(kc).flatten(-2), ks.to(torch.uint8)
            st["vc"][page, :, at], st["vs"][page, :, at] = packed(vc).flatten(-2), vs.to(torch.uint8)
        return tuple(decoded(st[c + "c"][page, :, at], st[c + "s"][page, :, at]).bfloat16() for c in "kv")
    # attention: sequences and their new tokens padded to the longest
    b, hkv, g, d = st["batch"], st["hkv"], st["hq"] // st["hkv"], st["d"]
    dev = st["q"].device
    key = torch.arange(st["max_len"], device=dev)
    page = st["table"][:, key // st["page"]].long()
    k, v = (decoded(st[c + "c"][page, :, key % st["page"]], st[c + "s"][page, :, key % st["page"]]).transpose(1, 2) for c in "kv")
    valid = key[None, :] < st["lens"][:, None]
    k, v = (torch.where(valid[:, None, :, None], t, torch.zeros((), device=dev)) for t in (k, v))
    seq, i = rows_of(st)
    q = torch.zeros(b, st["max_new"], hkv * g, d, device=dev)
    q[seq, i] = st["q"].float()
    q = q.view(b, -1, hkv, g, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    seen = valid[:, None, :].expand(-1, st["max_new"], -1)
    if st["causal"]:
        seen = seen & (key[None, None, :] <= (st["starts"][:, None] + torch.arange(st["max_new"], device=dev))[:, :, None])
    s.view(b, hkv, g, st["max_new"], -1).masked_fill_(~seen[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    y = (s @ v) / s.sum(-1, keepdim=True)
    y = y.view(b, hkv, g, st["max_new"], d).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return y[seq, i].bfloat16()


def seen_pairs(case):
    """(query token, key) pairs that the attention's mask leaves, and the cached positions that any query sees."""
    past, new = lengths(case)
    pairs = sum(n * p + (n * (n + 1) // 2 if case["causal"] else n * n) for p, n in zip(past, new))
    return pairs, sum(past) + sum(new)


def work(case):
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k // 2 + n * (k // 32) + m * n * (4 if case["f32"] else 2), "flops": 2 * m * n * k}
    past, new = lengths(case)
    row = 2 * case["hkv"] * case["d"]  # values of one position, keys and values
    held = row * 17 // 32  # their codes and scales
    if case["op"] == "read":
        return {"bytes": sum(past) * (held + 2 * row), "flops": sum(past) * row}
    if case["op"] == "cache":
        return {"bytes": sum(new) * ((4 if case["f32"] else 2) * row + held + 2 * row), "flops": 4 * sum(new) * row}
    pairs, keys = seen_pairs(case)
    return {"bytes": keys * held + 2 * 2 * sum(new) * case["hq"] * case["d"], "flops": 4 * pairs * case["hq"] * case["d"]}


# --- the same from the definitions, in 64 bits -------------------------------------------------------------------------------------------


def exact_values(codes, scales):
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=codes.device) / 2
    lo, hi = codes.long() % 16, codes.long() // 16
    n = torch.stack((lo, hi), dim=-1).reshape(*codes.shape[:-1], -1)
    v = mag[n % 8] * (1 - 2 * (n // 8)).double()
    return v * torch.pow(2.0, (scales.long() - 127).double()).repeat_interleave(32, dim=-1)


def exact_round(x):
    """Each block of 32 to the MXFP4 values nearest to it, by comparing with all of them."""
    x = x.double().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp_min(2.0 ** -140)))
    e = torch.where(torch.pow(2.0, e) > top, e - 1, e)
    e = torch.where(torch.pow(2.0, e + 1) <= top, e + 1, e)
    step = torch.pow(2.0, (e - 2).clamp(-127, 127))
    mag = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    a = (x / step).abs()
    best, near = torch.zeros_like(a), torch.full_like(a, math.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):  # the even codes first: they keep the ties
        off = (a - mag[c]).abs()
        best, near = torch.where(off < near, mag[c], best), torch.minimum(near, off)
    return (torch.copysign(best, x) * step).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        u = st["sf"].view(-1, (k // 32 + 3) // 4, 32, 4, 4)  # row group, block group, row % 32, row / 32 % 4, block % 4
        s = u.permute(0, 3, 2, 1, 4).reshape(u.shape[0] * 128, -1)[:n, :k // 32]
        return torch.cat([st["x"].double() @ exact_values(st["codes"][i:i + 1024], s[i:i + 1024]).T for i in range(0, n, 1024)], 1)
    past, new = lengths(case)
    if case["op"] == "cache":
        return tuple(torch.cat([exact_round(st[c][i:i + 2048].float()) for i in range(0, st["rows"], 2048)]) for c in "kv")
    outs, at = [], 0
    for b, (p, n) in enumerate(zip(past, new)):
        pages = st["table"][b, :(p + n + case["page"] - 1) // case["page"]].long()
        flat = lambda t: t[pages].transpose(1, 2).flatten(0, 1)[:p + n]  # noqa: E731
        kc, ks, vc, vs = (flat(st[t]) for t in ("kc", "ks", "vc", "vs"))
        if case["op"] == "read":
            outs.append((exact_values(kc, ks), exact_values(vc, vs)))
            continue
        g = case["hq"] // case["hkv"]
        y = torch.empty(n, case["hq"], case["d"], dtype=torch.float64, device=kc.device)
        for h in range(case["hkv"]):
            k, v = exact_values(kc[:, h], ks[:, h]), exact_values(vc[:, h], vs[:, h])
            for j in range(h * g, h * g + g):
                s = st["q"][at:at + n, j].double() @ k.T / math.sqrt(case["d"])
                if case["causal"]:
                    s = s.masked_fill(torch.arange(p + n, device=s.device)[None] > p + torch.arange(n, device=s.device)[:, None], -math.inf)
                y[:, j] = torch.softmax(s, -1) @ v
        outs.append(y)
        at += n
    if case["op"] == "read":
        return tuple(torch.cat(t) for t in zip(*outs))
    return torch.cat(outs)
