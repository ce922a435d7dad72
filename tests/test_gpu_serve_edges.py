"""The few-token operators where their ranges end: tables, batches, value ranges, streams.

Inputs and 64-bit forms are those of test_gpu_serve.py and serve_ref.py.
"""
import threading
import time

import pytest
import torch

import serve_ref as ref
import w4a4_mxfp4_post_b200 as kq
from test_gpu_serve import Plan, attend, normal, operand, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["native", "python"])
def either_binding(request, monkeypatch):
    """For what the binding does: its native part, and the Python calls."""
    if request.param == "python":
        monkeypatch.setattr(kq, "_native", lambda: False)
    else:
        assert kq._native(), "the binding's native part is not built"


def test_tables_whose_rows_share_memory_are_refused(cuda_device, either_binding):
    """An expanded table would be read past its end; its copy is taken."""
    p = Plan([40, 40, 40], [2, 2, 2], 2, 64, 16, seed=1)
    p.table = p.table[:1].expand(3, -1)
    q = normal(6, 8, 64, key=1)
    before = [t.clone() for t in p.cache]
    for table in (p.table, p.table[0].as_strided((3, p.table.shape[1]), (1, 1))):
        with pytest.raises(ValueError, match="overlap"):
            kq.mx_paged_attention(q, *p.cache, table, p.cud, p.lensd)
        with pytest.raises(ValueError, match="overlap"):
            kq.mx_cache_read(*p.cache, table, p.cud, 6)
        with pytest.raises(ValueError, match="overlap"):
            kq.mx_cache_write(q[:, :2], q[:, 2:4], *p.cache, table, p.cud, p.lensd)
    assert all(torch.equal(a, b) for a, b in zip(before, p.cache))
    p.table = p.table.contiguous()
    attend(p, q, max_new=2)


def test_a_single_sequence_with_any_row_stride(cuda_device, either_binding):
    p = Plan([70], [3], 2, 64, 16, seed=2)
    q = normal(3, 8, 64, key=2)
    want = attend(p, q, max_new=3)
    for stride in (0, 1, 1000):
        p.table = p.table.as_strided(p.table.shape, (stride, 1))
        assert torch.equal(attend(p, q, max_new=3), want)


# --- products ----------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 7, 12, 20])
@pytest.mark.parametrize("lo,hi", [(220, 227), (231, 241), (248, 255)])
def test_gemv_scales_up_to_the_largest(cuda_device, M, lo, hi):
    """Scales up to 2^127, beside the smallest ones in the same tile of weights, over rows of x of unlike sizes: every product
    whose terms fp32 holds comes out within its bound, with no infinity or NaN on the way."""
    N, K = 200, 1120
    c, s = operand(N, K, lo, lo, hi)
    g = rng(M, lo)
    small = torch.randint(0, 40, s.shape, dtype=torch.uint8, device="cuda", generator=g)
    kind = torch.arange(N, device="cuda") % 3
    s = torch.where(kind[:, None] == 0, small, s)            # all small, all large, and both within a row
    mixed = (kind[:, None] == 2) & (torch.rand(s.shape, device="cuda", generator=g) < 0.5)
    s = torch.where(mixed, small, s)
    gain = 2.0 ** torch.tensor([-(hi - 127) - 1 + 110, -(hi - 127) + 90, -90, 0, 20], device="cuda").float()
    x = (normal(M, K, key=lo).float() * gain[torch.arange(M, device="cuda") % 5][:, None]).bfloat16()
    y, ab, tail = ref.gemv(x, c, s)
    out = kq.mxf4_gemv(x, c, ref.sf_of(s), out_dtype=torch.float32)
    held = ab < 2.0 ** 126
    assert held.sum() > M * N // 4 and ((s >= 224).any(1)[None] & held & (ab > 2.0 ** 60)).any()
    # (2^-126: a rounding below fp32's normal numbers, as in test_gpu_serve.py)
    tol = ref.gemv_bound(y, ab, tail, K, False) + 2.0 ** -126
    assert ((out.double() - y).abs() <= tol)[held].all()


@pytest.mark.parametrize("M", [1, 20])
def test_gemv_of_one_and_a_large_weight(cuda_device, M):
    """x = 1 times a weight of 2^113 is 2^113."""
    N, K = 40, 256
    c = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    c[:, 5] = 2
    s = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    s[:, 0] = 240
    x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    assert (kq.mxf4_gemv(x, c, ref.sf_of(s)) == 2.0 ** 113).all()
    s[7, 0], s[9, 1] = 255, 255
    out = kq.mxf4_gemv(x, c, ref.sf_of(s))
    nan = torch.zeros(N, dtype=torch.bool, device="cuda")
    nan[[7, 9]] = True
    assert out[:, nan].isnan().all() and (out[:, ~nan] == 2.0 ** 113).all()


# --- attention ---------------------------------------------------------------

# a few rows (groups of 4 and 12: both widths); items that one CTA holds, and items that are split
LARGE = [([0], [1], 4), ([150], [1], 12), ([700, 90], [2, 1], 4), ([20000], [1], 4), ([9000, 12000], [3, 1], 4)]


def large_values(past, new, group, lo, hi, codes=None):
    p = Plan(past, new, 2, 64, 32, seed=lo)
    p.vs.copy_(torch.randint(lo, hi, p.vs.shape, dtype=torch.uint8, device="cuda", generator=rng(lo, hi)))
    if codes is not None:
        p.vc.fill_(codes)
    attend(p, normal(p.T, 2 * group, 64, key=lo), max_new=max(new))


@pytest.mark.parametrize("lo,hi,codes", [(225, 227, 0x77), (238, 246, None), (200, 253, None), (252, 253, 0x77), (252, 253, 0xF7)])
@pytest.mark.parametrize("past,new,group", LARGE)
def test_attention_values_up_to_the_largest(cuda_device, past, new, group, lo, hi, codes):
    """Sums over many positions of the largest values are past fp32, their mean is not."""
    large_values(past, new, group, lo, hi, codes)


# many rows: one tile and two, whole items and split ones, beside a single token's sequence
LARGE_CHUNKS = [([150], [64], 2), ([0], [300], 4), ([9000], [100], 4), ([2500, 500, 40], [90, 130, 1], 4)]


@pytest.mark.parametrize("lo,hi,codes", [(205, 211, None), (225, 227, 0x77), (238, 246, None), (200, 253, None), (252, 253, 0x77), (252, 253, 0xF7)])
@pytest.mark.parametrize("past,new,group", LARGE_CHUNKS)
def test_chunk_values_up_to_the_largest(cuda_device, past, new, group, lo, hi, codes):
    large_values(past, new, group, lo, hi, codes)
    assert kq.kq_wait_timeouts() == 0


@pytest.mark.parametrize("past", [0, 130, 3000])
def test_a_large_value_changes_nothing_for_who_does_not_see_it(cuda_device, past):
    """One token of a chunk has values near the end of the range: the rows before it keep their bits, those after it are right."""
    new, at = 150, 70
    p = Plan([past], [new], 2, 64, 32, seed=past)
    q = normal(new, 8, 64, key=past)
    base = attend(p, q, max_new=new)
    pos = past + at
    p.vs[int(p.table[0, pos // 32]), :, pos % 32] = 250
    out = attend(p, q, max_new=new)
    assert torch.equal(out[:at], base[:at]) and not torch.equal(out[at:], base[at:])


@pytest.mark.parametrize("top", [1, 13, 15, 16, 20, 25])
@pytest.mark.parametrize("past,new,group", [([0], [1], 4), ([150], [1], 12), ([9000], [1], 4), ([150], [64], 2), ([3000], [130], 4)])
def test_attention_values_of_the_smallest_scale(cuda_device, past, new, group, top):
    """Values of scale byte 0 (2^-127) beside zeros of larger scale bytes: 6 x 2^-127 is a normal number of bf16."""
    p = Plan(past, new, 2, 64, 32, seed=top)
    p.vc.fill_(0x77)
    p.vs.zero_()
    pos = torch.arange(0, p.lens[0], 3, device="cuda")
    pg, at = p.table[0][pos // 32].long(), pos % 32
    if past != [0]:
        p.vs[pg, :, at], p.vc[pg, :, at] = top, 0
    q = normal(p.T, 2 * group, 64, key=top)
    got = kq.mx_paged_attention(q, *p.args, max_new=max(new)).double()
    want, tol = ref.attention(q, p.cache, p.table, p.cu, p.lens, 64 ** -0.5, True)
    # where the weight of the zeros leaves less than 2^-126, bf16's steps are 2^-133 whatever the value: half a step of that
    assert ((got - want).abs() <= tol + 2.0 ** -134).all()
    assert (got != 0).any()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("past,new,group", [([0, 0], [1, 1], 4), ([60, 0], [1, 2], 12), ([9000, 16], [1, 1], 4), ([70, 0], [60, 40], 2), ([6000, 100], [100, 130], 4)])
def test_attention_of_infinite_queries(cuda_device, past, new, group, sign):
    """An infinity in a query makes each score that the row sees infinite: of one sign (-infinity for all of them, too) or NaN where
    the key is zero.  All that is NaN in the result, but zeros for a row that sees nothing, and no other row is touched."""
    p = Plan(past, new, 2, 64, 16, seed=sum(past))
    q = normal(p.T, 2 * group, 64, key=sum(new))
    p.lensd[1] = 0 if past[1] == 0 else p.lensd[1]
    base = attend(p, q, max_new=max(new))
    p.kc[:] = torch.where(p.kc & 7 == 0, p.kc | 1, p.kc) & 0x77               # no key code is negative
    p.kc[:] = torch.where(p.kc & 0x70 == 0, p.kc | 0x10, p.kc)                # or zero
    bad = q.clone()
    hit = torch.zeros(p.T, 2 * group, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[-1, 0] = hit[p.T // 2, group] = True
    bad[hit, 7] = sign * float("inf")
    out = attend(p, bad, max_new=max(new))
    sees = torch.tensor([p.lensd.tolist()[0 if t < new[0] else 1] > 0 for t in range(p.T)], device="cuda")
    assert torch.equal(out.isnan(), (hit & sees[:, None])[:, :, None].expand_as(out))
    assert (out[~sees] == 0).all() and (base[~sees] == 0).all()
    # zeros among the keys: NaN scores
    p.kc.zero_()
    attend(p, bad, max_new=max(new))


def test_attention_of_infinite_queries_over_holes(cuda_device):
    """A row is zero where its table names no page, whatever the query; NaN from the first page that it sees."""
    for new in (1, 70):
        p = Plan([100, 100], [new, new], 1, 64, 16, seed=new)
        p.table[0, :] = -1
        p.table[1, :3] = p.pages
        p.kc.fill_(0x22)
        q = normal(p.T, 4, 64, key=new)
        base = attend(p, q, max_new=new)
        q[:, 2, 9] = -float("inf")               # (the reference has no bound for such a row that sees nothing)
        out = kq.mx_paged_attention(q, *p.args, max_new=new)
        assert (out[:new] == 0).all() and out[new:, 2].isnan().all() and torch.equal(out[:, [0, 1, 3]], base[:, [0, 1, 3]])


@pytest.mark.parametrize("past,new,group", [([150], [1], 4), ([9000], [2], 8), ([200], [60], 4)])
def test_attention_of_a_large_scale_over_small_scores(cuda_device, past, new, group):
    """The scale is any finite number: 2^120 over products of 2^-150, whose scores are next to zero."""
    p = Plan(past, new, 2, 64, 32, seed=11)
    p.ks.copy_(torch.randint(60, 68, p.ks.shape, dtype=torch.uint8, device="cuda", generator=rng(11)))
    q = (normal(p.T, 2 * group, 64, key=11).float() * 2.0 ** -100).bfloat16()
    attend(p, q, scale=2.0 ** 120, max_new=max(new))


# --- the binding ---------------------------------------------------------------

def test_a_full_launch_queue_stops_no_other_thread(cuda_device, either_binding):
    """A call whose launch waits for a place in the queue waits without the interpreter's lock."""
    p = Plan([100], [1], 2, 64, 16, seed=3)
    x = normal(1, 16, 64, key=3)
    w, wsf = kq.mx_quantize_f32(torch.randn(64, 512, device="cuda"), sf_layout=True)
    calls = [lambda: kq.mx_cache_write(x[:, :2], x[:, 2:4], *p.args), lambda: kq.mx_cache_read(*p.cache, p.table, p.cud, 1),
             lambda: kq.mxf4_gemv(x.view(2, 512), w, wsf), lambda: kq.mx_paged_attention(x[:, 4:12], *p.args, max_new=1)]
    for call in calls:
        call()
        torch.cuda.synchronize()
        gaps, stop = [], threading.Event()

        def ticks():
            last = time.perf_counter()
            while not stop.is_set():
                time.sleep(0.001)
                now = time.perf_counter()
                gaps.append(now - last)
                last = now

        t = threading.Thread(target=ticks)
        t.start()
        torch.cuda._sleep(1_200_000_000)     # 0.6 s and more
        begun = time.perf_counter()
        for _ in range(2500):
            call()
        took = time.perf_counter() - begun
        torch.cuda.synchronize()
        stop.set()
        t.join()
        assert took > 0.3, "the queue did not fill"
        assert max(gaps) < 0.2, f"another thread stood still for {max(gaps):.2f} s"


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("op", ["gemv", "read", "attention"])
def test_results_of_another_stream_take_no_memory_of_the_current_one(cuda_device, op, raw):
    """Memory freed on the current stream is still read there; a call on another stream must not write it."""
    side = torch.cuda.Stream()
    p = Plan([0], [4096], 8, 128, 64, seed=4)
    x = normal(4096, 32, 128, key=4)
    w, wsf = kq.mx_quantize_f32(torch.randn(40000, 512, device="cuda"), sf_layout=True)
    call = {"gemv": lambda s: kq.mxf4_gemv(x.view(-1, 512)[:32], w, wsf, out_dtype=torch.float32, stream=s),
            "read": lambda s: kq.mx_cache_read(*p.cache, p.table, p.cud, 4096, stream=s)[0],
            "attention": lambda s: kq.mx_paged_attention(x, *p.args, max_new=4096, stream=s)}[op]
    want = call(None)
    call(side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    used = torch.full_like(want, 3.0)
    torch.cuda._sleep(200_000_000)           # 0.1 s: the copy below is still to come
    copy = used.clone()
    del used
    out = call(side.cuda_stream if raw else side)
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert (copy == 3).all()


def test_one_token_or_head_with_any_stride(cuda_device, either_binding):
    """Strides of dimensions of size 1 are not used, whatever the tensor says."""
    for H, new, st, sh in ((2, 1, 1331, None), (1, 3, None, 7), (1, 1, 5, 3)):
        p = Plan([20], [new], H, 64, 16, seed=6)
        k, v, q = (normal(new, H, 64, key=i) for i in (1, 2, 3))
        odd = [t.as_strided(t.shape, (st or t.stride(0), sh or t.stride(1), 1)) for t in (k, v, q)]
        copies = [[t.clone() for t in p.cache] for _ in range(2)]
        kq.mx_cache_write(k, v, *copies[0], p.table, p.cud, p.lensd)
        kq.mx_cache_write(*odd[:2], *copies[1], p.table, p.cud, p.lensd)
        assert all(torch.equal(a, b) for a, b in zip(*copies))
        assert torch.equal(kq.mx_paged_attention(odd[2], *p.args, max_new=new), kq.mx_paged_attention(q, *p.args, max_new=new))


# --- batches -------------------------------------------------------------------

@pytest.mark.parametrize("B", [63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("group", [4, 12])
def test_attention_of_large_batches_of_single_tokens(cuda_device, B, group):
    """As many sequences as threads that divide the work, fewer and more, ragged, some without tokens or length."""
    past = [(37 * b * b) % 211 for b in range(B)]
    new = [0 if b % 11 == 5 else 1 for b in range(B)]
    past[B // 2], past[B - 2] = 3000, 1700
    p = Plan(past, new, 2, 32, 16, seed=B)
    p.lensd[7] = 0
    attend(p, normal(p.T, 2 * group, 32, key=B), max_new=1)


@pytest.mark.parametrize("B", [129, 256, 257, 511, 513, 700])
def test_attention_of_large_batches_with_chunks(cuda_device, B):
    """Both kernels at once over such batches: sequences with more rows than the few-rows kernel takes beside single tokens."""
    past = [(53 * b * b) % 157 for b in range(B)]
    new = [(1, 7, 0, 2, 13)[b % 5] for b in range(B)]
    past[B // 3], new[B // 3] = 2500, 40
    p = Plan(past, new, 1, 32, 16, seed=B, pad=2)
    attend(p, normal(p.T, 8, 32, key=B), max_new=max(new))
    assert kq.kq_wait_timeouts() == 0


def test_cache_of_a_large_batch(cuda_device):
    """A single token for each of 1000 sequences, written and read back."""
    B = 1000
    p = Plan([b % 70 for b in range(B)], [1] * B, 2, 64, 16, seed=12)
    x = normal(B, 4, 64, key=12)
    kq.mx_cache_write(x[:, :2], x[:, 2:], *p.args)
    starts = torch.tensor(p.past, dtype=torch.int32, device="cuda")
    for got, src in zip(kq.mx_cache_read(*p.cache, p.table, p.cud, B, starts=starts), (x[:, :2], x[:, 2:])):
        codes, scales = kq.mx_quantize(src.reshape(2 * B, 64).contiguous())
        assert torch.equal(got.double(), ref.decode(codes, scales).view(B, 2, 64))


def test_chunks_repeat_bit_for_bit(cuda_device):
    p = Plan([3000, 20, 900], [90, 300, 1], 2, 128, 64, seed=13)
    q = normal(p.T, 16, 128, key=13)
    a = kq.mx_paged_attention(q, *p.args, max_new=300)
    assert all(torch.equal(a, kq.mx_paged_attention(q, *p.args, max_new=300)) for _ in range(4))
