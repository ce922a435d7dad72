"""The few-token operators against plain 64-bit forms: products with 4-bit
weights, the paged MXFP4 cache, attention over it, and a run of them together.

The bounds are derived in tests/serve_ref.py; codes and scale bytes are exact.
"""
import numpy as np
import pytest
import torch

import oracle
import serve_ref as ref
import w4a4_mxfp4_post_b200 as kq
from w4a4_mxfp4_post_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=["native", "python"])
def binding(request, monkeypatch):
    """Every test through both ways of the binding: its native part, and the Python calls."""
    if request.param == "python":
        monkeypatch.setattr(kq, "_native", lambda: False)
    else:
        assert kq._native(), "the binding's native part is not built"

NAN = float("nan")


def rng(*key):
    g = torch.Generator(device="cuda")
    return g.manual_seed(hash(key) % (1 << 31))


def operand(rows, K, seed, lo=112, hi=142):
    c, s = synth.mx_operand(rows, K, seed, lo, hi)
    return torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()


def normal(*shape, key=0, dtype=torch.bfloat16, spread=0.5):
    g = rng(shape, key)
    x = torch.randn(*shape, device="cuda", generator=g) * torch.exp(spread * torch.randn(shape[-1], device="cuda", generator=g))
    return x.to(dtype)


# --- products with a few rows -------------------------------------------------

GEMV = [(1, 1, 32), (1, 7, 64), (2, 130, 96), (3, 129, 4608), (4, 64, 160), (5, 5600, 2240), (8, 1152, 1152), (9, 300, 288),
        (13, 2240, 5600), (16, 128, 128), (17, 257, 1120), (24, 1000, 416), (32, 96, 4608), (32, 4608, 1152), (1, 20000, 256),
        (7, 33, 33 * 32), (1, 16, 40000), (31, 515, 8224)]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", GEMV, ids=["x".join(map(str, s)) for s in GEMV])
def test_gemv_matches_64_bits(cuda_device, M, N, K, f32):
    c, s = operand(N, K, M + N)
    x = normal(M, K, key=N)
    y, ab, tail = ref.gemv(x, c, s)
    dtype = torch.float32 if f32 else torch.bfloat16
    buf = torch.full((M * N + 64,), 7.0, dtype=dtype, device="cuda")
    out = kq.mxf4_gemv(x, c, ref.sf_of(s), out=buf[:M * N].view(M, N))
    assert ((out.double() - y).abs() <= ref.gemv_bound(y, ab, tail, K, not f32)).all()
    assert (buf[M * N:] == 7).all()


def test_gemv_reads_strided_rows_and_nothing_between(cuda_device):
    M, N, K = 6, 200, 1120
    c, s = operand(N, K, 5)
    wide = torch.full((M, K + 24), NAN, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + K] = normal(M, K, key=1)
    x = wide[:, 8:8 + K]
    assert torch.equal(kq.mxf4_gemv(x, c, ref.sf_of(s)), kq.mxf4_gemv(x.contiguous(), c, ref.sf_of(s)))


def test_gemv_zero_and_one_code_picks_single_elements(cuda_device):
    """Weights with a single code: every (row, element) comes out exactly, whatever its place in a tile."""
    N, K = 160, 352
    c = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    at = torch.randint(0, K, (N,), device="cuda", generator=rng(3))
    code = torch.randint(1, 16, (N,), device="cuda", generator=rng(4))
    r = torch.arange(N, device="cuda")
    c[r, at // 2] = torch.where(at % 2 == 0, code, code * 16).to(torch.uint8)
    x = normal(5, K, key=9)
    mag = torch.tensor(ref.MAG + tuple(-m for m in ref.MAG), device="cuda")
    want = x.float()[:, at] * mag[code]
    assert torch.equal(kq.mxf4_gemv(x, c, ref.sf_of(s), out_dtype=torch.float32), want)


@pytest.mark.parametrize("lo,hi", [(0, 3), (1, 60), (60, 200), (200, 230)])
def test_gemv_scales_over_the_whole_range(cuda_device, lo, hi):
    """Scales from the smallest up: fp32 holds these products, so the sums do too."""
    M, N, K = 3, 140, 256
    c, s = operand(N, K, 8, lo, hi)
    x = normal(M, K, key=2) * 2.0 ** (100 if hi <= 60 else 0)
    y, ab, tail = ref.gemv(x, c, s)
    out = kq.mxf4_gemv(x, c, ref.sf_of(s), out_dtype=torch.float32)
    tol = ref.gemv_bound(y, ab, tail, K, False) + 2.0 ** -126
    assert ((out.double() - y).abs() <= tol).all()


def test_gemv_rows_of_unlike_sizes(cuda_device):
    """x from bf16 subnormals to its top, zeros, and within one block 2^30 apart."""
    N, K = 70, 224
    c, s = operand(N, K, 11, 120, 130)
    x = normal(8, K, key=5).float()
    x[0] = 0
    x[1] *= 2.0 ** -130
    x[2] *= 2.0 ** 100
    x[3, ::2] *= 2.0 ** 30
    x[4, 32:64] *= 2.0 ** -60
    x[5] = -x[5] * 2.0 ** 60
    x = x.bfloat16()
    y, ab, tail = ref.gemv(x, c, s)
    out = kq.mxf4_gemv(x, c, ref.sf_of(s), out_dtype=torch.float32)
    tol = ref.gemv_bound(y, ab, tail, K, False) + 2.0 ** -126
    assert ((out.double() - y).abs() <= tol).all()
    assert (out[0] == 0).all()


def test_gemv_nan_and_infinity_stay_in_their_rows(cuda_device):
    M, N, K = 9, 150, 320
    c, s = operand(N, K, 12)
    x = normal(M, K, key=6)
    base = kq.mxf4_gemv(x, c, ref.sf_of(s), out_dtype=torch.float32)
    s2 = s.clone()
    s2[17, 3] = 255
    s2[149, 9] = 255
    out = kq.mxf4_gemv(x, c, ref.sf_of(s2), out_dtype=torch.float32)
    hit = torch.zeros(N, dtype=torch.bool, device="cuda")
    hit[[17, 149]] = True
    assert out[:, hit].isnan().all() and torch.equal(out[:, ~hit], base[:, ~hit])
    x2 = x.clone()
    x2[4, 100] = NAN
    x2[7, 3] = float("inf")
    out = kq.mxf4_gemv(x2, c, ref.sf_of(s), out_dtype=torch.float32)
    keep = [i for i in range(M) if i not in (4, 7)]
    assert out[4].isnan().all() and torch.equal(out[keep], base[keep])
    # infinity times a code: that sign's infinity, NaN where the code is zero
    code = (c[:, 1] >> 4) & 15
    zero, neg = (code & 7) == 0, code >= 8
    assert out[7][zero].isnan().all()
    assert (out[7][~zero] == torch.where(neg[~zero], -float("inf"), float("inf"))).all()


def test_gemv_same_weights_as_the_w4a4_product(cuda_device):
    """One copy of quantized weights serves both products: on a 4-bit activation they agree."""
    M, N, K = 16, 192, 1152
    w, wsf = kq.mx_quantize_f32(torch.randn(N, K, device="cuda", generator=rng(7)), sf_layout=True)
    x = normal(M, K, key=3)
    a, asc = kq.mx_quantize(x)
    xq = kq.mx_dequantize(a, asc).bfloat16()
    full = kq.mxf4_gemm(a, kq.mx_scales_to_sf(asc), w, wsf, out_dtype=torch.float32)
    few = kq.mxf4_gemv(xq, w, wsf, out_dtype=torch.float32)
    ws = torch.from_numpy(np.ascontiguousarray(oracle.mx_quantize_f32(torch.randn(N, K, device="cuda", generator=rng(7)).cpu().numpy())[1])).cuda()
    y, ab, tail = ref.gemv(xq, w, ws)
    tol = ref.gemv_bound(y, ab, tail, K, False)
    assert ((few.double() - y).abs() <= tol).all() and ((full.double() - y).abs() <= tol).all()


# --- the cache ------------------------------------------------------------------

class Plan:
    """A pool of pages and sequences in it: tables, lengths and rows, with a few pages of no sequence and junk everywhere."""

    def __init__(self, past, new, H, d, page, pad=0, seed=0, extra=3, junk=True, table_pad=0):
        self.past, self.new, self.H, self.d, self.page = past, new, H, d, page
        self.lens = [p + n for p, n in zip(past, new)]
        need = [(n + page - 1) // page for n in self.lens]
        self.pages = sum(need) + extra
        g = rng(seed, H, d, page)
        order = torch.randperm(self.pages, device="cuda", generator=g).int()
        wide = max(need + [1])
        full = torch.full((len(past), wide + table_pad), -7, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            full[b, :n] = order[at:at + n]
            at += n
        self.table = full[:, :wide]
        self.free = order[at:]
        self.cu = [sum(new[:i]) for i in range(len(new) + 1)]
        self.T = self.cu[-1] + pad
        self.cud = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        self.lensd = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        shape = (self.pages, H, page)
        self.kc, self.vc = (torch.randint(0, 256, (*shape, d // 2), dtype=torch.uint8, device="cuda", generator=g) for _ in "kv")
        self.ks, self.vs = (torch.randint(120, 128, (*shape, d // 32), dtype=torch.uint8, device="cuda", generator=g) for _ in "kv")
        if junk:
            # whatever no sequence holds: stale bytes, NaN scales among them
            used = torch.zeros(shape[0], page, dtype=torch.bool, device="cuda")
            for b, n in enumerate(self.lens):
                pos = torch.arange(n, device="cuda")
                used[self.table[b][pos // page].long(), pos % page] = True
            stale = ~used[:, None, :, None].expand(-1, H, -1, d // 32)
            for t in (self.ks, self.vs):
                t[stale] = torch.randint(250, 256, t.shape, dtype=torch.uint8, device="cuda", generator=g)[stale]

    @property
    def cache(self):
        return self.kc, self.ks, self.vc, self.vs

    @property
    def args(self):
        return (*self.cache, self.table, self.cud, self.lensd)


def bits(x):
    return np.ascontiguousarray(x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


def quantized(x):
    """Codes and scales of [T, H, d] by the oracle."""
    T, H, d = x.shape
    if T == 0:
        return (torch.zeros(0, H, d // 2, dtype=torch.uint8), torch.zeros(0, H, d // 32, dtype=torch.uint8))
    if x.dtype == torch.bfloat16:
        c, s = oracle.mx_quantize(bits(x).reshape(T * H, d))
    else:
        c, s = oracle.mx_quantize_f32(np.ascontiguousarray(x.contiguous().cpu().numpy()).reshape(T * H, d))
    return torch.from_numpy(c).view(T, H, d // 2), torch.from_numpy(s).view(T, H, d // 32)


CACHES = [  # past, new, heads, d, page, padding rows
    ([0], [1], 1, 32, 16, 0),
    ([15], [1], 2, 64, 16, 0),
    ([16], [1], 2, 64, 16, 3),
    ([0, 5, 63, 200], [33, 1, 2, 0], 3, 96, 32, 5),
    ([7, 0, 0, 31], [0, 0, 70, 17], 4, 128, 48, 0),
    ([100] * 40, [1] * 40, 8, 128, 64, 24),
    ([0, 1000], [700, 300], 2, 128, 128, 1),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CACHES, ids=[f"{sum(c[1])}rows_d{c[3]}_p{c[4]}" for c in CACHES])
def test_cache_write_and_read(cuda_device, case, dtype):
    past, new, H, d, page, pad = case
    p = Plan(past, new, H, d, page, pad, table_pad=3)
    # keys and values as slices of a fused projection: query heads, then keys, then values
    qkv = normal(p.T, 2 + 2 * H, d, key=1, dtype=dtype)
    k, v = qkv[:, 2:2 + H], qkv[:, 2 + H:]
    want = [t.clone() for t in p.cache]
    (kc, ks), (vc, vs) = quantized(k), quantized(v)
    for b in range(len(new)):
        for i in range(new[b]):
            pos, t = past[b] + i, p.cu[b] + i
            pg = int(p.table[b, pos // page])
            for dst, src in zip(want, (kc, ks, vc, vs)):
                dst[pg, :, pos % page] = src[t].cuda()
    kq.mx_cache_write(k, v, *p.args)
    for got, w, name in zip(p.cache, want, ("k codes", "k scales", "v codes", "v scales")):
        assert torch.equal(got, w), name
    # read everything back
    cu = torch.tensor([sum(p.lens[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    rows = int(cu[-1]) + pad
    for f32 in (False, True):
        out = [torch.full((rows, H, d), 3.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda") for _ in "kv"]
        kq.mx_cache_read(*p.cache, p.table, cu, rows, out_k=out[0], out_v=out[1])
        for b in range(len(new)):
            for o, c, s in zip(out, (p.kc, p.vc), (p.ks, p.vs)):
                w, _ = ref.gather(c, s, p.table[b], p.lens[b], p.pages)
                assert torch.equal(o[int(cu[b]):int(cu[b + 1])].double(), w)
        assert all((o[int(cu[-1]):] == 3).all() for o in out)
    # and the new tokens alone
    starts = torch.tensor(past, dtype=torch.int32, device="cuda")
    ko, vo = kq.mx_cache_read(*p.cache, p.table, p.cud, p.cu[-1], starts=starts)
    assert torch.equal(ko.cpu().double(), ref.decode(kc, ks)[:p.cu[-1]])
    assert torch.equal(vo.cpu().double(), ref.decode(vc, vs)[:p.cu[-1]])


def test_cache_write_of_values_that_are_not_finite(cuda_device):
    p = Plan([0], [4], 2, 64, 16)
    k = normal(4, 2, 64, key=2)
    k[1, 0, 40] = NAN
    k[2, 1, 3] = -float("inf")
    kq.mx_cache_write(k, k, *p.args)
    pg = int(p.table[0, 0])
    assert p.ks[pg, 0, 1].tolist()[1] == 255 and p.ks[pg, 1, 2].tolist()[0] == 255
    assert (p.kc[pg, 0, 1, 16:] == 0).all()
    ko, _ = kq.mx_cache_read(*p.cache, p.table, p.cud, 4)
    nan = ko.isnan()
    assert nan.sum() == 64 and nan[1, 0, 32:].all() and nan[2, 1, :32].all()


def test_cache_skips_positions_on_no_page(cuda_device):
    """Table entries outside the pool, positions behind the table and before 0: nothing is written, zeros are read."""
    p = Plan([0, 0, 30], [40, 16, 20], 2, 64, 16, extra=4)
    p.table[0, 1] = -1
    p.table[1, 0] = p.pages
    p.table[2, 2] = 1 << 30
    p.lensd[1] = 3                     # 16 new tokens of a sequence of 3: 13 before position 0
    k = normal(p.T, 2, 64, key=4)
    want = [t.clone() for t in p.cache]
    c, s = quantized(k)
    for b, (n, ln) in enumerate(zip((40, 16, 20), p.lensd.tolist())):
        for i in range(n):
            pos, t = ln - n + i, p.cu[b] + i
            pg = int(p.table[b, pos // 16]) if pos >= 0 else -1
            if 0 <= pg < p.pages:
                for dst, src in zip(want, (c, s, c, s)):
                    dst[pg, :, pos % 16] = src[t].cuda()
    kq.mx_cache_write(k, k, *p.args)
    for got, w in zip(p.cache, want):
        assert torch.equal(got, w)
    cu = torch.tensor([0, 60, 70, 120], dtype=torch.int32, device="cuda")   # past the tables' ends
    ko, vo = kq.mx_cache_read(*p.cache, p.table, cu, 120)
    for b, (lo, hi) in enumerate(((0, 60), (60, 70), (70, 120))):
        w, _ = ref.gather(p.kc, p.ks, p.table[b], hi - lo, p.pages)
        # stale bytes among them: 4 * 2^126 and more (scale bytes 253, 254) is infinity in bf16
        assert torch.equal(torch.nan_to_num(ko[lo:hi], nan=-99.0), torch.nan_to_num(w.bfloat16(), nan=-99.0))
    # a table with no columns holds no position
    none = p.table[:, :0]
    before = [t.clone() for t in p.cache]
    kq.mx_cache_write(k, k, *p.cache, none, p.cud, p.lensd)
    assert all(torch.equal(a, b) for a, b in zip(before, p.cache))
    assert (kq.mx_cache_read(*p.cache, none, p.cud, p.T)[0] == 0).all()


# --- attention --------------------------------------------------------------------

def attend(p, q, causal=True, scale=None, out=None, **kw):
    """The call, checked against 64 bits; rows of no sequence keep their values."""
    T, hq, d = q.shape
    if out is None:
        out = torch.full((T, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    got = kq.mx_paged_attention(q, *p.args, causal=causal, scale=scale, out=out, **kw)
    want, tol = ref.attention(q, p.cache, p.table, p.cu, p.lensd.tolist(), d ** -0.5 if scale is None else scale, causal)
    n = p.cu[-1]
    assert (got[n:] == 5).all()
    g, w, t = got[:n].double(), want[:n], tol[:n]
    assert torch.equal(g.isnan(), w.isnan()), "NaN in other places"
    off = torch.where(w.isnan(), torch.zeros_like(w), (g - w).abs() - t)
    assert (off <= 0).all(), f"off by {float(off.max())} over its bound"
    return got


# past, new, kv heads, group, d, page, padding rows
ATTN = [
    ([0], [1], 1, 1, 32, 16, 0),
    ([15], [1], 1, 3, 64, 16, 2),
    ([16], [1], 2, 4, 64, 16, 0),
    ([127], [1], 2, 8, 128, 64, 0),
    ([128], [1], 2, 5, 96, 32, 0),
    ([1000, 3, 0, 517, 64], [1, 1, 1, 1, 1], 2, 4, 128, 64, 3),
    ([300] * 33, [1] * 33, 1, 8, 64, 48, 0),
    ([5000], [1], 1, 16, 128, 128, 0),
    ([9000, 100], [1, 1], 4, 1, 128, 64, 0),
    ([40, 0, 1000], [4, 2, 3], 2, 4, 128, 16, 1),
    ([100, 31], [5, 7], 1, 6, 96, 48, 0),
    ([0], [17], 2, 2, 32, 16, 0),
    ([0], [128], 2, 1, 64, 64, 0),
    ([0], [129], 1, 4, 128, 64, 0),
    ([77, 0, 1500], [130, 300, 1], 2, 4, 128, 64, 5),
    ([640], [257], 1, 3, 96, 32, 0),
    ([33, 2000], [64, 70], 2, 8, 64, 48, 0),
    ([4096], [200], 1, 8, 128, 128, 0),
    ([10], [500], 1, 1, 32, 16, 0),
    ([0, 0, 0, 0], [0, 33, 0, 65], 2, 4, 128, 16, 0),
]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
@pytest.mark.parametrize("case", ATTN, ids=["_".join(map(str, (f"b{len(c[0])}", max(c[0]), max(c[1]), f"h{c[2]}x{c[3]}", f"d{c[4]}", f"p{c[5]}"))) for c in ATTN])
def test_attention_matches_64_bits(cuda_device, case, causal):
    past, new, H, g, d, page, pad = case
    p = Plan(past, new, H, d, page, pad, seed=sum(past) + len(new), table_pad=2)
    q = normal(p.T, H * g, d, key=7)
    attend(p, q, causal, max_new=max(new))


@pytest.mark.parametrize("max_new", [None, 0, 1, 3, 40, 10000])
def test_attention_takes_any_bound_on_the_new_tokens(cuda_device, max_new):
    """max_new selects kernels; a mixed batch comes out right under any."""
    p = Plan([900, 40, 0, 333], [1, 40, 150, 3], 2, 128, 64, 2, seed=5)
    attend(p, normal(p.T, 8, 128, key=8), max_new=max_new)


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 0.02])
def test_attention_scales(cuda_device, new, scale):
    p = Plan([200], [new], 2, 64, 32, seed=6)
    attend(p, normal(p.T, 8, 64, key=9), scale=scale, max_new=new)


@pytest.mark.parametrize("new", [1, 100])
def test_attention_reads_strided_queries(cuda_device, new):
    p = Plan([333], [new], 2, 128, 64, seed=7)
    wide = torch.full((new, 20, 128), NAN, dtype=torch.bfloat16, device="cuda")
    wide[:, 5:13] = normal(new, 8, 128, key=10)
    a = attend(p, wide[:, 5:13], max_new=new)
    b = attend(p, wide[:, 5:13].contiguous(), max_new=new)
    assert torch.equal(a, b)
    by_head = wide[:, 5:13].transpose(0, 1).contiguous().transpose(0, 1)      # [heads][tokens] in memory
    assert torch.equal(attend(p, by_head, max_new=new), b)


@pytest.mark.parametrize("new", [1, 5, 140])
def test_attention_rows_that_see_nothing(cuda_device, new):
    """Sequences of no length or shorter than their new tokens, tables with holes and without pages: zeros, and other rows as they are."""
    p = Plan([100, 70, 64, 50], [new] * 4, 2, 64, 16, seed=8)
    p.lensd[0] = 0
    p.lensd[1] = new // 2
    p.table[2, :] = -1
    p.table[3, 1] = p.pages + 3
    q = normal(p.T, 4, 64, key=11)
    for causal in (True, False):
        out = attend(p, q, causal, max_new=new)
        assert (out[:new] == 0).all() and (out[2 * new:3 * new] == 0).all()
    p.lensd[0] = -5
    attend(p, q, True, max_new=new)


@pytest.mark.parametrize("new", [1, 4, 150])
def test_attention_nan_reaches_only_who_sees_it(cuda_device, new):
    """NaN blocks among the keys and the values, seen by all rows, by the later ones, or by none (the reference masks by position)."""
    for what in ("k", "v"):
        p = Plan([300, 40, 200], [new] * 3, 2, 128, 32, seed=9)
        c, s = (p.kc, p.ks) if what == "k" else (p.vc, p.vs)
        for b, pos, h, j, byte in ((0, 17, 0, 2, 255), (1, 40 + new // 2, 1, 0, 255), (1, 40 + new - 1, 0, 3, 254), (0, 299, 1, 1, 253)):
            pg = int(p.table[b, pos // 32])
            s[pg, h, pos % 32, j] = byte
            c[pg, h, pos % 32, 16 * j:16 * j + 16] = 0 if byte == 255 else 0x11
        q = normal(p.T, 8, 128, key=12)
        for causal in (True, False):
            out = attend(p, q, causal, max_new=new)
            assert out.isnan().any() and not out[2 * new:].isnan().any()


@pytest.mark.parametrize("new", [1, 120])
def test_attention_of_nan_and_infinite_queries(cuda_device, new):
    p = Plan([100, 60], [new, new], 1, 64, 16, seed=10)
    q = normal(p.T, 4, 64, key=13)
    base = attend(p, q, max_new=new)
    bad = q.clone()
    bad[0, 1, 5] = NAN
    out = kq.mx_paged_attention(bad, *p.args, max_new=new)
    keep = torch.ones(p.T, 4, dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert out[0, 1].isnan().all() and torch.equal(out[keep], base[keep])


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("lo,hi", [(0, 3), (20, 24), (126, 134), (150, 160), (180, 186)])
def test_attention_values_of_any_size(cuda_device, new, lo, hi):
    """Value scales over the format's range, and tokens of unlike sizes side by side."""
    p = Plan([150], [new], 2, 128, 32, seed=lo)
    p.vs.copy_(torch.randint(lo, hi, p.vs.shape, dtype=torch.uint8, device="cuda", generator=rng(lo, hi)))
    p.ks.copy_(torch.randint(115, 122, p.ks.shape, dtype=torch.uint8, device="cuda", generator=rng(lo)))
    q = normal(p.T, 8, 128, key=14)
    got = kq.mx_paged_attention(q, *p.args, max_new=new).double()
    want, tol = ref.attention(q, p.cache, p.table, p.cu, p.lens, 128 ** -0.5, True)
    assert ((got - want).abs() <= tol + 2.0 ** -126).all()


@pytest.mark.parametrize("new", [1, 64])
def test_attention_of_unlike_tokens(cuda_device, new):
    """Value scales 60 binades apart within a sequence, the rows' weight on the small ones: the large ones' weight is not lost in rounding, nor the small ones."""
    p = Plan([200], [new], 1, 64, 16, seed=21)
    n = p.lens[0]
    pos = torch.arange(n, device="cuda")
    pg, at = p.table[0][pos // 16].long(), pos % 16
    p.vs[pg, :, at] = torch.where(pos % 7 == 3, 167, 107).to(torch.uint8)[:, None, None]
    # keys: a constant direction, large where the values are small
    p.kc[pg, :, at] = 0x22
    p.ks[pg, :, at] = torch.where(pos % 7 == 3, 1, 128).to(torch.uint8)[:, None, None]
    for s in (0.1, 0.5, 0.7):
        q = torch.ones(new, 4, 64, dtype=torch.bfloat16, device="cuda")
        attend(p, q, scale=s, max_new=new)


@pytest.mark.parametrize("new", [1, 64])
def test_attention_keys_and_queries_of_any_size(cuda_device, new):
    for lo, hi, gain in ((5, 9, 2.0 ** 119), (240, 244, 2.0 ** -117), (60, 64, 2.0 ** 64), (190, 194, 2.0 ** -66)):
        p = Plan([150], [new], 2, 64, 16, seed=lo)
        p.ks.copy_(torch.randint(lo, hi, p.ks.shape, dtype=torch.uint8, device="cuda", generator=rng(lo, hi)))
        q = (normal(p.T, 4, 64, key=15).float() * gain).bfloat16()
        attend(p, q, max_new=new)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_scores_far_apart(cuda_device, new):
    """Scores that grow along the sequence (the maximum moves all the way) and that fall (the first is all)."""
    p = Plan([700], [new], 1, 64, 32, seed=16)
    n = p.lens[0]
    pos = torch.arange(n, device="cuda")
    pg, at = p.table[0][pos // 32].long(), pos % 32
    p.kc[pg, :, at] = 0x22                                                   # all ones
    p.ks[pg, :, at] = (110 + pos // 40).to(torch.uint8)[:, None, None]
    for sign in (1.0, -1.0):
        q = torch.full((new, 2, 64), sign * 4, dtype=torch.bfloat16, device="cuda")
        attend(p, q, max_new=new)


def test_attention_with_group_of_many_heads(cuda_device):
    for g in (24, 40, 64, 100):
        p = Plan([210, 15], [1, 2], 1, 64, 16, seed=g)
        attend(p, normal(p.T, g, 64, key=g), max_new=2)


def test_attention_shared_pages(cuda_device):
    """Two sequences that share the pages of a common prefix."""
    p = Plan([128, 128], [20, 9], 2, 64, 32, seed=17)
    p.table[1, :4] = p.table[0, :4]
    attend(p, normal(p.T, 8, 64, key=17), max_new=20)


def test_attention_repeats_bit_for_bit(cuda_device):
    """The work is split by the lengths alone: the same call gives the same bits, and a row's neighbours may only change the split."""
    p = Plan([3000, 200, 7000], [1, 1, 1], 2, 128, 64, seed=18)
    q = normal(3, 16, 128, key=18)
    a = kq.mx_paged_attention(q, *p.args, max_new=1)
    for _ in range(3):
        assert torch.equal(a, kq.mx_paged_attention(q, *p.args, max_new=1))


def test_caches_past_32_bit_offsets(cuda_device):
    """Pages whose bytes lie past 2^31 and 2^32 of the pool."""
    H, d, page = 8, 128, 128
    pages = (5 << 30) // (H * page * d // 2)
    kc = torch.empty(pages, H, page, d // 2, dtype=torch.uint8, device="cuda")
    ks = torch.empty(pages, H, page, d // 32, dtype=torch.uint8, device="cuda")
    far = [pages - 1, pages // 2 + 3, 1, pages - 3]
    table = torch.tensor([far], dtype=torch.int32, device="cuda")
    for new in (1, 100):
        n = 3 * page + 30
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        k = normal(n, H, d, key=new)
        kq.mx_cache_write(k, k, kc, ks, kc, ks, table, cu, lens)
        ko, vo = kq.mx_cache_read(kc, ks, kc, ks, table, cu, n)
        c, s = quantized(k)
        assert torch.equal(ko.cpu().double(), ref.decode(c, s)) and torch.equal(ko, vo)
        q = normal(new, H, d, key=3)
        cq = torch.tensor([0, new], dtype=torch.int32, device="cuda")
        got = kq.mx_paged_attention(q, kc, ks, kc, ks, table, cq, lens, max_new=new)
        sel = torch.tensor(far, device="cuda")
        small = (kc[sel], ks[sel], kc[sel], ks[sel])
        want, tol = ref.attention(q, small, torch.arange(4, dtype=torch.int32, device="cuda")[None], [0, new], [n], d ** -0.5, True)
        assert ((got.double() - want).abs() <= tol).all()


# --- streams, graphs ----------------------------------------------------------------

def test_calls_on_another_stream(cuda_device):
    p = Plan([900, 100], [1, 60], 2, 128, 64, seed=19)
    q = normal(p.T, 8, 128, key=19)
    want = kq.mx_paged_attention(q, *p.args, max_new=60)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        out = torch.zeros_like(want)
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            kq.mx_paged_attention(q, *p.args, max_new=60, out=out, stream=stream)
            # memory of the default stream's pool that is written at once must not be the call's workspace
            junk = torch.full((1 << 22,), NAN, device="cuda")
        side.synchronize()
        assert torch.equal(out, want) and junk.isnan().all()


def test_two_captured_graphs_and_eager_calls(cuda_device):
    """A whole step (write, attention, product) captured twice over different inputs, replayed in turn and beside eager calls; lengths change between replays."""
    H, g, d, page, N = 2, 4, 64, 16, 200
    steps = []
    w, wsf = kq.mx_quantize_f32(torch.randn(N, H * g * d, device="cuda", generator=rng(20)), sf_layout=True)
    for i in range(2):
        p = Plan([100 + 60 * i, 40], [1, 1], H, d, page, seed=30 + i, extra=8)
        steps.append((p, normal(2, H * g + 2 * H, d, key=40 + i)))

    def step(p, x):
        k, v = x[:, H * g:H * g + H], x[:, H * g + H:]
        kq.mx_cache_write(k, v, *p.args)
        o = kq.mx_paged_attention(x[:, :H * g], *p.args, max_new=1)
        return o, kq.mxf4_gemv(o.view(2, -1), w, wsf)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for p, x in steps:
            step(p, x)
    torch.cuda.synchronize()
    graphs = []
    for p, x in steps:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = step(p, x)
        graphs.append((gr, res))
    for r in range(3):
        for p, x in steps:
            x.copy_(normal(*x.shape, key=100 + r))
            p.lensd += 1 if r else 0               # the next token's place (both tables have pages for it)
        want = [[t.clone() for t in step(p, x)] for p, x in steps]
        for gr, _ in graphs:
            gr.replay()
        for (gr, res), ww in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(res, ww))


# --- together -------------------------------------------------------------------------

@pytest.mark.parametrize("transformed", [False, True], ids=["plain", "kroquant"])
def test_a_layer_answers_token_by_token(cuda_device, transformed):
    """A prompt, then single tokens, through cache, attention and output product against
    64 bits.  With the KroQuant transform, keys are stored as T k (kq_transform_f32) and
    queries enter as q T^-1 (kq_fold_weights), which leaves every q . k as it was: the
    reference attends over the decoded cache with the same queries."""
    H, g, d, page, N = 2, 4, 64, 16, 256
    hq = H * g
    p = Plan([0, 0], [0, 0], H, d, page, extra=24, seed=50)
    p.table = p.free[:24].view(2, 12)[:, :11].contiguous()
    lens = [0, 0]
    w, wsf = kq.mx_quantize_f32(torch.randn(N, hq * d, device="cuda", generator=rng(51)), sf_layout=True)
    wc, ws = oracle.mx_quantize_f32(torch.randn(N, hq * d, device="cuda", generator=rng(51)).cpu().numpy())
    ws = torch.from_numpy(ws).cuda()
    F = torch.from_numpy(synth.factors(d // 32, 3)).cuda()
    for step, new in enumerate(((37, 90), (1, 1), (1, 1), (3, 0), (1, 1), (20, 1))):
        cu = [0, new[0], new[0] + new[1]]
        T = cu[-1]
        lens = [a + b for a, b in zip(lens, new)]
        p.cu, p.cud = cu, torch.tensor(cu, dtype=torch.int32, device="cuda")
        p.lens, p.lensd = lens, torch.tensor(lens, dtype=torch.int32, device="cuda")
        x = normal(T, hq + 2 * H, d, key=60 + step)
        q, k, v = x[:, :hq], x[:, hq:hq + H], x[:, hq + H:]
        if transformed:
            k = kq.kq_transform_f32(k.reshape(T * H, d), F).view(T, H, d)
            q = kq.kq_fold_weights(q.float().reshape(T * hq, d), F).view(T, hq, d).bfloat16()
            v = v.float().contiguous()
        kq.mx_cache_write(k, v, *p.args)
        o = attend(p, q, max_new=max(new))
        if T > 32:
            continue
        y = kq.mxf4_gemv(o.view(T, hq * d), w, wsf, out_dtype=torch.float32)
        want, ab, tail = ref.gemv(o.view(T, hq * d), w, ws)
        assert ((y.double() - want).abs() <= ref.gemv_bound(want, ab, tail, hq * d, False)).all()
    assert kq.kq_wait_timeouts() == 0


@pytest.mark.parametrize("hkv,new", [(8, 32), (40, 20), (8, 70), (3, 150)])
def test_attention_items_of_one_and_two_tiles_in_turn(cuda_device, hkv, new):
    """Many heads whose rows end in a half-filled item, long contexts beside short ones: no wait of the kernels runs out."""
    p = Plan([1500, 0, 130], [new, new, new // 2], hkv, 64, 16, seed=70)
    attend(p, normal(p.T, 4 * hkv, 64, key=70), max_new=new)
    assert kq.kq_wait_timeouts() == 0


def test_a_pool_without_pages_holds_nothing(cuda_device):
    """No pages at all: nothing is written, zeros are read and attended."""
    kc, ks = torch.empty(0, 2, 16, 32, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, 16, 2, dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    for new in (1, 40):
        cu, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, new], [new]))
        x = normal(new, 4, 64, key=new)
        kq.mx_cache_write(x[:, :2], x[:, 2:], kc, ks, kc, ks, table, cu, lens)
        assert (kq.mx_cache_read(kc, ks, kc, ks, table, cu, new)[1] == 0).all()
        assert (kq.mx_paged_attention(x, kc, ks, kc, ks, table, cu, lens) == 0).all()


def test_calls_side_by_side(cuda_device):
    """Chunks, single tokens, products of both kinds on streams of their own at once, each with its own workspace."""
    plans = [Plan([900, 30], [200, 90], 2, 128, 64, seed=80), Plan([2000] * 5, [1] * 5, 2, 128, 64, seed=81),
             Plan([100], [300], 4, 64, 16, seed=82)]
    qs = [normal(p.T, 4 * p.H, p.d, key=83) for p in plans]
    w, wsf = kq.mx_quantize_f32(torch.randn(3000, 2048, device="cuda", generator=rng(84)), sf_layout=True)
    xs = [normal(m, 2048, key=m) for m in (3, 12, 30)]
    a, asc = kq.mx_quantize(normal(256, 2048, key=85))
    a_sf = kq.mx_scales_to_sf(asc)
    want = [kq.mx_paged_attention(q, *p.args, max_new=max(p.new)) for p, q in zip(plans, qs)] + [kq.mxf4_gemv(x, w, wsf) for x in xs]
    want.append(kq.mxf4_gemm(a, a_sf, w, wsf))
    torch.cuda.synchronize()
    outs = [torch.zeros_like(t) for t in want]
    streams = [torch.cuda.Stream() for _ in want]
    work = [torch.empty(kq.mx_attention_workspace(p.T, 4 * p.H, p.H, p.d, max(p.new)), dtype=torch.uint8, device="cuda") for p in plans]
    work += [torch.empty(kq.mxf4_gemv_workspace(x.shape[0], 3000, 2048), dtype=torch.uint8, device="cuda") for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            if i < 3:
                kq.mx_paged_attention(qs[i], *plans[i].args, max_new=max(plans[i].new), out=outs[i], workspace=work[i], stream=s)
            elif i < 6:
                kq.mxf4_gemv(xs[i - 3], w, wsf, out=outs[i], workspace=work[i], stream=s)
            else:
                kq.mxf4_gemm(a, a_sf, w, wsf, out=outs[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want)) and kq.kq_wait_timeouts() == 0


def test_captured_chunks_and_converted_products(cuda_device):
    """A chunk over a cache and a product that converts its rows beforehand, captured twice and replayed over new inputs."""
    N, K, M = 700, 1024, 24
    w, wsf = kq.mx_quantize_f32(torch.randn(N, K, device="cuda", generator=rng(90)), sf_layout=True)
    steps = [(Plan([500 + i, 60], [70, 33], 2, 64, 16, seed=91 + i), normal(103, 8, 64, key=92 + i), normal(M, K, key=94 + i)) for i in range(2)]

    def step(p, q, x):
        return kq.mx_paged_attention(q, *p.args, max_new=70), kq.mxf4_gemv(x, w, wsf)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for s in steps:
            step(*s)
    torch.cuda.synchronize()
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step(*s)
        graphs.append((g, res))
    for r in range(3):
        for p, q, x in steps:
            q.copy_(normal(*q.shape, key=200 + r))
            x.copy_(normal(*x.shape, key=300 + r))
        want = [[t.clone() for t in step(*s)] for s in steps]
        for g, _ in graphs:
            g.replay()
        for (_, res), ww in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(res, ww))
    assert kq.kq_wait_timeouts() == 0


def test_attention_of_wide_value_ranges_among_ordinary_ones(cuda_device):
    """Stages whose value scales lie further apart than fp16 takes beside stages that do not, zero blocks and the smallest scales among them."""
    for spread in (6, 12, 13, 14, 40, 126):
        p = Plan([1500], [2], 2, 128, 32, seed=spread)
        pos = torch.arange(p.lens[0], device="cuda")
        pg, at = p.table[0][pos // 32].long(), pos % 32
        p.vs[pg, :, at] = 127
        low = (pos // 64) % 3 == 1
        p.vs[pg[low], :, at[low]] = 127 - spread
        p.vs[pg[pos % 50 == 7], :, at[pos % 50 == 7], 1] = 0
        attend(p, normal(p.T, 8, 128, key=spread), max_new=2)


def test_native_binding_leaves_the_unusual_to_python(cuda_device):
    """Wrong types and shapes are refused with the same errors either way; subclasses and strided tables work."""
    p = Plan([40], [3], 2, 64, 16, seed=95, table_pad=4)
    q = normal(3, 8, 64, key=95)
    want = kq.mx_paged_attention(q, *p.args, max_new=3)
    assert torch.equal(kq.mx_paged_attention(torch.nn.Parameter(q, requires_grad=False), *p.args), want)

    class Sub(torch.Tensor):
        pass

    assert torch.equal(kq.mx_paged_attention(q.as_subclass(Sub), *p.args).as_subclass(torch.Tensor), want)
    with pytest.raises(TypeError):
        kq.mx_paged_attention(q.float(), *p.args)
    with pytest.raises(TypeError):
        kq.mx_paged_attention(q, *p.cache, p.table.long(), p.cud, p.lensd)
    with pytest.raises(ValueError):
        kq.mx_paged_attention(q, *p.cache, p.table, p.cud[:1], p.lensd)
    with pytest.raises(ValueError):
        kq.mx_paged_attention(q[:, :3], *p.args)
    with pytest.raises(ValueError):
        kq.mx_paged_attention(q, *p.args, max_new=-1)
    with pytest.raises(kq.KroQuantError):
        kq.mx_paged_attention(q, *p.args, scale=float("inf"))
    with pytest.raises(TypeError):
        kq.mx_paged_attention(q, *p.cache, p.table, p.cud, None)
    with pytest.raises(ValueError):
        kq.mx_cache_write(q, q, *p.args)
    with pytest.raises(TypeError):
        kq.mx_cache_write(q[:, :2], q[:, 2:4].float(), *p.args)
    with pytest.raises((ValueError, RuntimeError)):
        kq.mx_cache_read(*p.cache, p.table, p.cud, -1)
    w, wsf = kq.mx_quantize_f32(torch.randn(64, 512, device="cuda"), sf_layout=True)
    x = normal(5, 512, key=96)
    assert torch.equal(kq.mxf4_gemv(x, w, wsf, out_dtype=torch.float32).bfloat16(), kq.mxf4_gemv(x, w, wsf))
    with pytest.raises(ValueError):
        kq.mxf4_gemv(x[:, :256], w, wsf)
    with pytest.raises(ValueError):
        kq.mxf4_gemv(x, w, wsf[:-1])
    with pytest.raises(kq.KroQuantError):
        kq.mxf4_gemv(normal(33, 512, key=97), w, wsf)
