// mx_attention.cuh -- attention of a chunk of new tokens over a paged MXFP4
// cache.  Included by kroquant.cu; uses its helpers, mx_cache.cuh and
// mxf4_gemv.cuh.
//
//   out[t][h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[t][h] . k_j - max)
//
// over the positions j of t's sequence that its mask leaves: j <= the
// position of t (causal) or every j below the sequence's length.  Positions
// whose page the table does not name are not seen.  A row that sees nothing
// is zero, one that sees nothing but scores of -infinity NaN.
//
// Work.  The query heads of a kv head and the new tokens of a sequence are the
// rows of one product over that head's cache: row r of (sequence b, kv head h)
// is token r / g, query head h g + r % g.  An item is R consecutive rows of one
// (b, h); it takes ceil(end / 128) units of 128 positions, end being the last
// position that any of its rows sees.  The units of all items, in order, are
// dealt out in equal contiguous shares to a grid that fills the GPU once, from
// the lengths on the device: no plan on the host, ragged batches balance, and
// long sequences split over as many CTAs as they need.  (What an item costs beside
// its units counts as units, too: a causal prompt of 4096, whose first items are
// one unit long, took 253 us without, 165 with.)  A CTA whose share ends inside
// an item leaves a partial result (maximum, sum, output of its positions alone)
// in its slot of the workspace, and merge_kernel adds up the partials of the
// items that were split, in order: the same lengths give the same bits.
// (Partial outputs are weighted means, as the result: sums over many positions of
// values near the end of the format's range are past that of fp32.)

namespace attn {

constexpr int kUnit = 128;                   // positions per unit of work
constexpr int kMaxCtas = 512;                // shares (the workspace has two slots for each)
constexpr int kWindow = 12;                  // binades of value scales that fp16 products take together
constexpr uint32_t kNanByte = 253;           // K and V scale bytes from here up read as NaN

struct Args {
    const __nv_bfloat16 *q;
    int64_t q_st, q_sh;                      // strides of a token and a head (elements)
    const uint8_t *kc, *ks, *vc, *vs;
    __nv_bfloat16 *out;                      // [T][hq][D]
    float scale_log2;                        // scale * log2(e)
    int causal;
    int hq, group;                           // query heads, query heads per kv head
    int rows_lo, rows_hi;                    // sequences with rows_lo < rows <= rows_hi are this kernel's
    int page_shift;                          // log2(page), -1 if it is no power of two
    uint8_t *work;                           // workspace
    cache::Seqs s;
};

// What a CTA left behind: the item that its share ended in, if the item began
// there and goes on (parts > 0: that many shares hold it, this one the first).
struct Desc {
    int parts;
    int h, r0;                               // kv head, first row
    int lo, rows;                            // the sequence's first row of the call, its rows
    int b;                                   // sequence
    int pad[2];
};

// Slot i of a workspace for R rows: output [D / 4][R][4] (a thread per row writes
// whole lines), maxima [R], sums [R].
template <int R, int D>
__device__ __forceinline__ float *slot(const Args &a, int i)
{
    return reinterpret_cast<float *>(a.work + kMaxCtas * sizeof(Desc)) + int64_t(i) * R * (D + 2);
}

template <int R>
__device__ __forceinline__ int slot_at(int row, int d) { return ((d >> 2) * R + row) * 4 + (d & 3); }

// A sequence as the kernels see it.
struct Seq {
    int lo, n, len, rows;                    // first row of the call, new tokens, length, rows per kv head
};

__device__ __forceinline__ Seq load_seq(const Args &a, int b)
{
    Seq q;
    int hi;
    cache::seq_rows(a.s, b, q.lo, hi);
    q.n = hi - q.lo;
    q.len = __ldg(a.s.len + b);
    q.rows = q.n * a.group;
    if (q.rows <= a.rows_lo || q.rows > a.rows_hi) q.rows = 0;
    return q;
}

// Positions that row r sees: [0, row_end).
__device__ __forceinline__ int row_end(const Args &a, const Seq &q, int r)
{
    const int64_t e = a.causal ? int64_t(q.len) - q.n + r / a.group + 1 : q.len;
    return int(max(int64_t(0), min(e, cache::seq_cap(a.s))));
}

// Units of the item with rows tile * R ..; at least one, which writes the rows
// that see nothing.
template <int R>
__device__ __forceinline__ int item_units(const Args &a, const Seq &q, int tile)
{
    return max(1, (row_end(a, q, min((tile + 1) * R, q.rows) - 1) + kUnit - 1) / kUnit);
}

// What an item costs beside its units (queries, results, filling the pipeline)
// counts as V units before its first: shares are cut in units and these.
template <int R, int V>
__device__ __forceinline__ int64_t head_cost(const Args &a, const Seq &q)
{
    const int tiles = (q.rows + R - 1) / R;
    if (!a.causal) return int64_t(tiles) * (tiles ? item_units<R>(a, q, 0) + V : 0);
    int64_t u = 0;
    for (int t = 0; t < tiles; ++t) u += item_units<R>(a, q, t) + V;
    return u;
}

// x / y of numbers that are not negative: in 32 bits where they are that small,
// for a division of 64 takes hundreds of clocks.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y)
{
    return ((x | y) >> 32) == 0 ? int64_t(uint32_t(x) / uint32_t(y)) : x / y;
}

// A place in the order of units: sequence, head, tile, unit of the item.
struct Place {
    int b, h, tile, unit;
};

// The share of this CTA: its first unit's place and its cost from there on (none
// if it holds no unit).  There are `shares` of them, one for each CTA but no more
// than units, so that every share between an item's first and last holds a part
// of it.  Every thread of
// the CTA calls it; `sh` is shared memory of THREADS + 34 int64.  The threads
// count a head's units: of one sequence's tiles each (as many threads to a
// sequence as there are), or of several sequences.
template <int R, int V, int THREADS>
__device__ __forceinline__ int64_t my_share(const Args &a, int64_t *sh, Place &p, int64_t &total, int &shares)
{
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int split = a.s.B < THREADS ? THREADS / max(a.s.B, 1) : 1;         // threads of a sequence
    const int per = (a.s.B + THREADS - 1) / THREADS;                         // or sequences of a thread
    const int b0 = min(split > 1 ? tid / split : tid * per, a.s.B), b1 = split > 1 ? min(b0 + 1, a.s.B) : min(b0 + per, a.s.B);
    auto first_tile = [&](int rows, int part) {
        const int tiles = (rows + R - 1) / R, each = tiles / split;
        return part * each + min(part, tiles - each * split);
    };
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        const Seq q = load_seq(a, b);
        const int part = split > 1 ? tid % split : 0, t1 = first_tile(q.rows, part + 1);
        int t = first_tile(q.rows, part);
        if (a.causal)
            for (; t < t1; ++t) mine += item_units<R>(a, q, t) + V;
        else if (t < t1)
            mine += int64_t(t1 - t) * (item_units<R>(a, q, t) + V);
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
    }
    int64_t *sums = sh + THREADS;
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += sums[w];
    sh[tid] = incl;
    __syncthreads();
    total = sh[THREADS - 1] * a.s.heads;
    shares = int(min(int64_t(gridDim.x), total));
    if (int(blockIdx.x) >= shares) return 0;
    const int64_t first = quotient(total * blockIdx.x, shares);
    const int64_t last = quotient(total * (blockIdx.x + 1), shares);
    int *place = reinterpret_cast<int *>(sums + 32);
    const bool leads = b0 < b1 && (split == 1 || tid % split == 0);          // of its sequences' threads
    int64_t at = (incl - mine) * a.s.heads;                                  // units before its sequences
    if (leads && first >= at && first < sh[tid + split - 1] * a.s.heads) {
        int b = b0, t = 0, h;
        int64_t off = first - at;
        Seq q = load_seq(a, b);
        if (split > 1) {
            const int64_t before = incl - mine, hu = sh[tid + split - 1] - before;
            h = int(quotient(off, hu));
            off -= h * hu;
            int lo = 0, hi = split - 1;      // the part that holds the unit
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sh[tid + mid] - before > off) hi = mid;
                else lo = mid + 1;
            }
            if (lo > 0) off -= sh[tid + lo - 1] - before;
            t = first_tile(q.rows, lo);
        } else {
            int64_t hu = head_cost<R, V>(a, q);
            while (off >= hu * a.s.heads) {  // ends: the units of b0 .. b1 - 1 hold `first`
                off -= hu * a.s.heads;
                q = load_seq(a, ++b);
                hu = head_cost<R, V>(a, q);
            }
            h = int(quotient(off, hu));
            off -= h * hu;
        }
        for (int u = item_units<R>(a, q, t) + V; off >= u; u = item_units<R>(a, q, ++t) + V) off -= u;
        place[0] = b;
        place[1] = h;
        place[2] = t;
        place[3] = int(off);
    }
    __syncthreads();
    // (a share that begins within the V begins with the first unit)
    p = Place{place[0], place[1], place[2], max(place[3] - V, 0)};
    return last - first - max(V - place[3], 0);
}

// The share that unit u is in (counted with the V): the last i with total * i / shares <= u.
__device__ __forceinline__ int64_t share_of(int64_t u, int64_t total, int64_t shares)
{
    return quotient((u + 1) * shares + total - 1, total) - 1;
}

// The next item after (b, h, tile): tiles, then heads, then sequences that have rows.
template <int R>
__device__ __forceinline__ void next_item(const Args &a, Seq &q, Place &p)
{
    p.unit = 0;
    if (++p.tile * R < q.rows) return;
    p.tile = 0;
    if (++p.h < a.s.heads) return;
    p.h = 0;
    do {
        if (++p.b >= a.s.B) return;
        q = load_seq(a, p.b);
    } while (q.rows == 0);
}

// The first of the 16 pool rows that hold positions t .. t + 15 of sequence b's
// head h (t a multiple of 16 below the table's capacity), -1 if on no page.
__device__ __forceinline__ int64_t strip_row(const Args &a, const int32_t *table, int h, int t)
{
    const int j = a.page_shift >= 0 ? t >> a.page_shift : t / a.s.page;
    const int p = __ldg(table + j);
    if (p < 0 || p >= a.s.num_pages) return -1;
    return (int64_t(p) * a.s.heads + h) * a.s.page + (t - j * a.s.page);
}

// What a row of sequence b with a sum of zero is divided by the sum to: it saw
// nothing (zeros stay), or every score that it saw was -infinity (NaN).
__device__ __noinline__ float empty_row(const int32_t *table, int page, int num_pages, int end)
{
    for (int j = 0; int64_t(j) * page < end; ++j) {
        const int p = __ldg(table + j);
        if (p >= 0 && p < num_pages) return __uint_as_float(0x7fc00000u);
    }
    return 0.0f;
}

__device__ __forceinline__ float empty_row(const Args &a, int b, int end)
{
    return empty_row(a.s.table + int64_t(b) * a.s.table_stride, a.s.page, a.s.num_pages, end);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^e for any int e (0 below fp32's normal numbers, infinity above).
__device__ __forceinline__ float pow2(int e)
{
    return e < -126 ? 0.0f : __uint_as_float(uint32_t(min(e, 128) + 127) << 23);
}

// x * 2^e for -253 <= e <= 127, where 2^e itself may be below fp32's normal numbers.
__device__ __forceinline__ float times_pow2(float x, int e)
{
    const int most = max(e, -126);
    return x * pow2(most) * pow2(e - most);
}

// ---------------------------------------------------------------------------
// A few rows (R = 8 or 16): the cache streams through once.
//
// Bound: the cache's bytes, 17 per 32 values, against the issue slots and the
// ALU pipe (unpacking).  At 6.5 TB/s an SM sub-partition gets 16 positions of
// keys and values of 128 channels (2176 bytes) every 375 clocks.
//
// Both products are transposed, so that the rows are the 8-column operand of
// mma.m16n8k16 and nothing is padded to 16 rows:
//   S^T = K Q^T    16 positions x channels, times channels x 8 rows
//   O^T += V^T P^T 16 channels x 16 positions, times positions x 8 rows
// Keys are unpacked to fp16 by cvt (2 clocks per pair) without their scales;
// a 32-block's two MMAs run into zero and its scale is applied to the four
// sums in fp32, relative to the stage's largest.  q is brought to fp16 by a
// power of two per row that puts its largest element in [2^15, 2^16): exact
// down to 2^-32 of it, else off by at most 2^-40 of it.
// The values' scale varies along the summed dimension, so it has to be in an
// operand.  It goes into P, which is small: 2 multiplies per 32 channels and 16
// positions instead of one per pair of values.  Values are then plain fp16 codes
// (ldmatrix.trans brings 4 codes of two positions into a register, 6 bit
// operations pair up 16 codes, cvt unpacks them), and a 32-block of channels has
// its own P' = p 2^15 2^(scale - top) in fp16, top the warp's largest value scale
// so far: half a step, 2^-11 of each probability, or 2^-40 of the largest
// probability times the largest scale, whichever is more.  Stages where a scale
// lies more than 2^12 below top (rare) take bf16 instead, values expanded by
// shifts (the code's bits 8, 7, 6 and 15 are code * 2^-126, which one packed
// multiply by 2^(126 + scale - top) makes exact) and P in bf16.
// P^T leaves the first product with positions along the rows and enters the
// second along the columns: movmatrix transposes it.
//
// A CTA is four warps, each with its own softmax state and its own cp.async
// ring of stages (32 positions of keys, values and scales); a warp takes every
// fourth stage of the share and waits for nothing but its own copies.  They
// meet when an item ends.  Three CTAs to an SM: with four (128 registers) the
// shares get shorter (16 x 40000 took 199 us where three took 176, two steps ago).
//
// Outputs are kept relative to the largest value scale that the warp has seen and
// leave the kernel divided by their sum: neither 2^15 nor a sum over many
// positions takes values near the end of the format's range past fp32.
//
// Measured, 64 query heads over 8 of 128 channels: 16 sequences of 27 to 40
// thousand positions 165 us, 3.6 TB/s (0.55 of the copy bandwidth); 32 of 2.7 to
// 4 thousand 48 us.  Issue slots 54 % and ALU 51 % busy at 2.7 warps per
// scheduler: it is the instructions, some 670 per stage (1000 with values in
// bf16, scales byte by byte and the maximum by shuffles), that bound it.  A quarter
// of them unpack codes; about half are the stage's own (scales, votes, tables,
// maxima, addresses) whatever the channels and rows: 32 x 4096 takes 34, 39, 46 and
// 48 us with 32, 64, 96 and 128 channels.  With 9 to 16 rows (NT = 2) 128 channels
// spill, and more than 16 rows are items that read the cache again: 16 x 8000 with
// 32 rows 107 us, with 16 rows 67.
template <int D_, int NT_>
struct Few {
    static constexpr int D = D_, NT = NT_;
    static constexpr int R = 8 * NT;
    static constexpr int kWarps = 4;
    static constexpr int kItemCost = 1;                      // of an item beside its units, in units
    static constexpr int kMergeRows = 2;                     // rows that a CTA of the merge takes
    static constexpr int kStages = 3;
    static constexpr int NB = D / 32;
    static constexpr int MT = 2 * NB;                        // 16-channel tiles of O
    static constexpr int kRow = D >= 96 ? 64 : D / 2;        // bytes of a position's codes in the stage
    static constexpr int kBytes = 32 * kRow;                 // of keys or values
    static constexpr int kScaleBytes = 32 * NB;              // of keys; the values' follow
    static constexpr int kStage = 2 * kBytes + 2 * kScaleBytes;
    static constexpr int kTable = 32 * 4 * 4 + 16 * 4 * 4;   // key scales (fp32), value scales (16-bit pairs)
    static constexpr int kWarpBytes = kStages * kStage + kTable;
    static constexpr int kOutRow = D + 4;                    // floats
    static constexpr int kMerge = kWarps * R * (kOutRow + 2) * 4;
    static constexpr int kSmem = kWarps * kWarpBytes > kMerge ? kWarps * kWarpBytes : kMerge;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit elements over the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t hmul2_f16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four 8 x 8 matrices of 16-bit elements, transposed: with rows of 16 bytes of
// codes, register i holds codes 4 g .. 4 g + 3 of positions 2 c and 2 c + 1.
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Code p (0..3) of both 16-bit halves as bf16 values code * 2^-126: sign to bit
// 15, the three magnitude bits to the exponent's lowest two and the mantissa's
// highest, where 0.5 (code 1) is a subnormal.
template <int P>
__device__ __forceinline__ uint32_t code_bf16(uint32_t w)
{
    const uint32_t s = P < 3 ? w << (12 - 4 * P) : w;
    const uint32_t m = P < 2 ? w << (6 - 4 * P) : w >> (4 * P - 6);
    return (s & 0x80008000u) | (m & 0x01C001C0u);
}

template <class C>
__global__ void __launch_bounds__(C::kWarps * 32, 3)
few_kernel(const Args a)
{
    pdl_wait();
    constexpr int D = C::D, NT = C::NT, R = C::R, NB = C::NB, MT = C::MT, W = C::kWarps, ST = C::kStages;
    // (aligned to whole 32-byte sectors at least: on 16 bytes 16 x 40000 takes 8 % longer)
    extern __shared__ __align__(128) uint8_t smem_few[];
    __shared__ int64_t sh[W * 32 + 34];
    __shared__ int nan_first[4];             // per 32 channels: the first position of the item whose value is NaN
    __shared__ int vtops[W];                 // the warps' largest value scales
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;

    Place p;
    int64_t total;
    int shares;
    int64_t left = my_share<R, C::kItemCost, W * 32>(a, sh, p, total, shares);
    Desc *desc = reinterpret_cast<Desc *>(a.work) + blockIdx.x;
    if (threadIdx.x == 0) desc->parts = 0;
    if (left <= 0) return;

    uint8_t *ring = smem_few + warp * C::kWarpBytes;
    float *ktab = reinterpret_cast<float *>(ring + ST * C::kStage);          // [32 positions][4]
    uint32_t *vtab = reinterpret_cast<uint32_t *>(ktab + 128);               // [16 pairs][4]
    const uint32_t ring_s = smem_addr(ring);
    // ldmatrix: this lane's row of the strip (matrices: positions 0-7, 8-15 of two 32-blocks) and its swizzle
    const int vrow = lane & 15, vsw = D >= 96 ? (vrow >> 1) & 3 : D == 64 ? (vrow >> 2) & 1 : 0, vsel = lane >> 4;

    // Where piece i of a strip (chunk i % NB of row i / NB) goes: chunks xor-swizzled by row.  For NB a power of two
    // 32 pieces are 32 / NB rows, a multiple of 8, so the next ones have the same swizzle.
    auto place = [](int i) {
        const int r = i / NB, ch = i % NB;
        return r * C::kRow + (D >= 96 ? ch ^ ((r >> 1) & 3) : D == 64 ? ch ^ ((r >> 2) & 1) : ch) * 16;
    };
    const uint32_t place0 = place(lane);

    Seq q = load_seq(a, p.b);
    while (left > 0) {
        // ---- the segment: units [p.unit, p.unit + count) of item (b, h, tile)
        const int units = item_units<R>(a, q, p.tile);
        const int count = int(min(left, int64_t(units - p.unit)));
        const int r0 = p.tile * R;
        const int item_end = row_end(a, q, min(r0 + R, q.rows) - 1);
        const int t_end = min(item_end, (p.unit + count) * kUnit);
        const int32_t *table = a.s.table + int64_t(p.b) * a.s.table_stride;

        // q, then the first stages on their way before q is used (a small call 9.8 -> 9.0 us); a row that is not
        // there reads the last one's
        uint4 raw[NT][NB];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = min(r0 + 8 * t + g, q.rows - 1), token = r / a.group;
            const __nv_bfloat16 *from =
                a.q + int64_t(q.lo + token) * a.q_st + int64_t(p.h * a.group + r - token * a.group) * a.q_sh + 8 * c;
#pragma unroll
            for (int b = 0; b < NB; ++b) raw[t][b] = __ldg(reinterpret_cast<const uint4 *>(from + 32 * b));
        }
        uint32_t on_page = 0;                                // two bits per stage in flight: its strips have a page

        const int t_first = p.unit * kUnit + warp * 32;
        auto fetch = [&](int t0, int slot_i) {               // stage: positions t0 .. t0 + 31
            uint32_t bits = 0;
            if (t0 < t_end) {
                const uint32_t dst = ring_s + slot_i * C::kStage;
                int64_t row = -1;
#pragma unroll
                for (int s = 0; s < 2; ++s) {                // strips of 16 positions, contiguous in the pool
                    // (pages of 32 positions and more: a stage is on one)
                    if (s == 0 || a.page_shift < 5) row = t0 + 16 * s < t_end ? strip_row(a, table, p.h, t0 + 16 * s) : -1;
                    else row = row >= 0 && t0 + 16 < t_end ? row + 16 : -1;
                    const uint32_t size = row >= 0 ? 16 : 0;
                    bits |= row >= 0 ? 1u << s : 0u;
                    const int64_t at = row >= 0 ? row : 0;
                    const uint8_t *k = a.kc + at * (D / 2) + lane * 16, *v = a.vc + at * (D / 2) + lane * 16;
#pragma unroll
                    for (int j = 0; j < (NB + 1) / 2; ++j) { // 16 NB pieces, 32 at a time
                        if (NB % 2 == 0 || 32 * j + lane < 16 * NB) {
                            const uint32_t to = dst + 16 * s * C::kRow + (NB == 3 ? place(lane + 32 * j) : place0 + 32 / NB * j * C::kRow);
                            gemv::cp_async16_sized(to, k + 512 * j, size);
                            gemv::cp_async16_sized(to + C::kBytes, v + 512 * j, size);
                        }
                    }
                    if (lane < 2 * NB) {                     // scales: 16 NB bytes of a strip are contiguous
                        const bool is_v = lane >= NB;
                        const int piece = is_v ? lane - NB : lane;
                        gemv::cp_async16_sized(dst + 2 * C::kBytes + (is_v ? C::kScaleBytes : 0) + s * 16 * NB + piece * 16,
                                               (is_v ? a.vs : a.ks) + at * NB + piece * 16, size);
                    }
                }
            }
            gemv::cp_commit();
            on_page |= bits << (2 * (ST - 1));
        };

#pragma unroll
        for (int i = 0; i < ST - 1; ++i) {
            on_page >>= 2;
            fetch(t_first + i * 32 * W, i);
        }
        // q as the 8-column operand: fp16, a power of two per row
        uint32_t qf[NT][NB][4];
        int qexp[NT];                                        // of row 8 nt + g
        int lim[NT][2], lim_min = 0x7fffffff;                // of rows 8 nt + 2 c, + 1
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 8 * t + g;
            uint32_t top = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (r >= q.rows) raw[t][b] = make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w[4] = {raw[t][b].x, raw[t][b].y, raw[t][b].z, raw[t][b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {                // the largest finite magnitude: an infinity stays one
                    const uint32_t lo = (w[i] << 16) & 0x7fff0000u, hi = w[i] & 0x7fff0000u;
                    top = max(top, max(lo < 0x7f800000u ? lo : 0u, hi < 0x7f800000u ? hi : 0u));
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int field = max(int(top >> 23) - 15, 1);
            const float down = __uint_as_float(uint32_t(254 - field) << 23);
            qexp[t] = field - 127;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t w[4] = {raw[t][b].x, raw[t][b].y, raw[t][b].z, raw[t][b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[t][b][i] = gemv::pack_f16x2(bf16_lo(w[i]) * down, bf16_hi(w[i]) * down);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int rr = r0 + 8 * t + 2 * c + i;
                lim[t][i] = rr < q.rows ? row_end(a, q, rr) : 0;
                if (rr < q.rows) lim_min = min(lim_min, lim[t][i]);
            }
        }
        lim_min = __reduce_min_sync(0xffffffffu, lim_min);
        int qe[NT][2];                                       // exponents of rows 8 nt + 2 c, + 1
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) qe[t][i] = __shfl_sync(0xffffffffu, qexp[t], 8 * c + 4 * i);

        if (threadIdx.x < 4) nan_first[threadIdx.x] = 0x7fffffff;
        __syncthreads();

        float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.0f;
        }
        int vtop = 0, kref = 0;                              // the largest value and key scale bytes so far
        float cs[NT][2];                                     // what brings S to units of log 2
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) cs[t][i] = times_pow2(a.scale_log2, qe[t][i] - 127);
        int it = 0;
        for (int t0 = t_first; t0 < t_end; t0 += 32 * W, ++it) {
            gemv::cp_wait<ST - 2>();
            __syncwarp();
            on_page >>= 2;
            const uint32_t pages = on_page & 3;
            fetch(t0 + (ST - 1) * 32 * W, (it + ST - 1) % ST);
            const uint8_t *st = ring + (it % ST) * C::kStage;

            // ---- scales of the stage: lane = position
            const bool valid = t0 + lane < t_end && ((pages >> (lane >> 4)) & 1);
            const uint32_t mask = __ballot_sync(0xffffffffu, valid);
            // bytes 0, 2 and 1, 3 of the position's scales as 16-bit pairs (0 where it counts for nothing: its P is 0)
            uint32_t k2[2], v2[2];
            {
                const uint8_t *ks = st + 2 * C::kBytes + lane * NB;
                uint32_t wk = 0, wv = 0;
                if constexpr (NB == 4) {
                    wk = *reinterpret_cast<const uint32_t *>(ks);
                    wv = *reinterpret_cast<const uint32_t *>(ks + C::kScaleBytes);
                } else {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        wk |= uint32_t(ks[b]) << (8 * b);
                        wv |= uint32_t(ks[C::kScaleBytes + b]) << (8 * b);
                    }
                }
                wk = valid ? wk : 0u;
                wv = valid ? wv : 0u;
                k2[0] = wk & 0x00ff00ffu, k2[1] = (wk >> 8) & 0x00ff00ffu;
                v2[0] = wv & 0x00ff00ffu, v2[1] = (wv >> 8) & 0x00ff00ffu;
            }
            uint32_t knan = 0;                               // blocks of the position that are NaN
            {
                const uint32_t km = __vmaxu2(k2[0], k2[1]), vm = __vmaxu2(v2[0], v2[1]);
                if (__any_sync(0xffffffffu, max(km >> 16, km & 0xffffu) > uint32_t(kref) || max(vm >> 16, vm & 0xffffu) > uint32_t(vtop))) {
                    // rare but for the first stages: larger scales, and NaN (253 and more; such values count as zero here)
                    int ktop = 0, vmax = 0;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const int sh = 16 * (b >> 1), kb = (k2[b & 1] >> sh) & 0xff, vb = (v2[b & 1] >> sh) & 0xff;
                        if (kb >= int(kNanByte)) {
                            knan |= 1u << b;
                            k2[b & 1] &= ~(0xffu << sh);
                        } else {
                            ktop = max(ktop, kb);
                        }
                        if (vb >= int(kNanByte)) {
                            atomicMin(&nan_first[b], t0 + lane);
                            v2[b & 1] &= ~(0xffu << sh);
                        } else {
                            vmax = max(vmax, vb);
                        }
                    }
                    ktop = __reduce_max_sync(0xffffffffu, ktop);
                    if (ktop > kref) {
                        kref = ktop;
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i) cs[t][i] = times_pow2(a.scale_log2, min(qe[t][i] + kref - 127, 127));
                    }
                    vmax = __reduce_max_sync(0xffffffffu, vmax);
                    if (vmax > vtop) {
                        const float f = pow2(vtop - vmax);
                        vtop = vmax;
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int i = 0; i < MT; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[t][i][e] *= f;
                    }
                }
            }
            // a block with 0 < scale < vtop - kWindow: bit 8 of (scale + 255), and not of scale + 256 - the limit.  Scale
            // 0 is a block of zeros' (it counts for nothing in fp16) or 2^-127, which counts while that is not below
            // 2^-40 of the largest: up to 55.
            bool wide;
            {
                const uint32_t limit = uint32_t(256 - max(vtop - kWindow, 0)) * 0x00010001u;
                const uint32_t some = vtop < 56 ? 0x01000100u : 0x00ff00ffu;
                const uint32_t low = ((v2[0] + some) & ~(v2[0] + limit)) | ((v2[1] + some) & ~(v2[1] + limit));
                wide = __any_sync(0xffffffffu, (low & 0x01000100u) != 0);
            }
            {
                // exponents relative to the largest, by pairs: max(scale, ref - e0) - (ref - e0) is the field of 2^(scale - ref)
                // where e0 is that of 1, and 0 below
                auto fields = [](uint32_t x, int ref, int e0) {
                    return __vmaxu2(x, uint32_t(max(ref - e0, 0)) * 0x00010001u) + uint32_t(e0 - ref) * 0x00010001u;
                };
                const uint32_t k02 = fields(k2[0], kref, 127), k13 = fields(k2[1], kref, 127);
                float kv[4] = {__uint_as_float(k02 << 23), __uint_as_float(k13 << 23), __uint_as_float((k02 << 7) & 0x7f800000u),
                               __uint_as_float((k13 << 7) & 0x7f800000u)};
                if (knan)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if ((knan >> b) & 1) kv[b] = __uint_as_float(0x7fc00000u);
                *reinterpret_cast<float4 *>(ktab + 4 * lane) = make_float4(kv[0], kv[1], kv[2], kv[3]);
                // fp16 2^(scale - vtop) or bf16 2^(126 + scale - vtop); two positions to a word
                uint32_t f02, f13;
                if (!wide) {
                    f02 = fields(v2[0], vtop, 15) << 10;
                    f13 = fields(v2[1], vtop, 15) << 10;
                } else {
                    f02 = (v2[0] + uint32_t(253 - vtop) * 0x00010001u) << 7;
                    f13 = (v2[1] + uint32_t(253 - vtop) * 0x00010001u) << 7;
                }
                const uint32_t sel = lane & 1 ? 0x3276u : 0x5410u;
                const uint32_t w0 = __byte_perm(f02, __shfl_xor_sync(0xffffffffu, f02, 1), sel);
                const uint32_t w1 = __byte_perm(f13, __shfl_xor_sync(0xffffffffu, f13, 1), sel);
                *reinterpret_cast<uint2 *>(vtab + (lane >> 1) * 4 + (lane & 1) * 2) = make_uint2(w0, w1);
            }
            __syncwarp();

            // ---- S^T: rows 16 s + g, + 8; columns 8 t + 2 c, + 1
            float s[2][NT][4];
#pragma unroll
            for (int sp = 0; sp < 2; ++sp) {
#pragma unroll
                for (int t = 0; t < NT; ++t) s[sp][t][0] = s[sp][t][1] = s[sp][t][2] = s[sp][t][3] = 0.0f;
                const float4 f0 = *reinterpret_cast<const float4 *>(ktab + 4 * (16 * sp + g));
                const float4 f1 = *reinterpret_cast<const float4 *>(ktab + 4 * (16 * sp + g + 8));
                const float k0[4] = {f0.x, f0.y, f0.z, f0.w}, k1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int ch = D >= 96 ? b ^ ((g >> 1) & 3) : D == 64 ? b ^ ((g >> 2) & 1) : b;
                    const uint8_t *kr = st + (16 * sp + g) * C::kRow + ch * 16 + 4 * c;
                    uint32_t x[4], y[4];
                    gemv::codes_f16(*reinterpret_cast<const uint32_t *>(kr), x);
                    gemv::codes_f16(*reinterpret_cast<const uint32_t *>(kr + 8 * C::kRow), y);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        gemv::mma_f16(z, x[0], y[0], x[1], y[1], qf[t][b][0], qf[t][b][1]);
                        gemv::mma_f16(z, x[2], y[2], x[3], y[3], qf[t][b][2], qf[t][b][3]);
                        s[sp][t][0] = fmaf(z[0], k0[b], s[sp][t][0]);
                        s[sp][t][1] = fmaf(z[1], k0[b], s[sp][t][1]);
                        s[sp][t][2] = fmaf(z[2], k1[b], s[sp][t][2]);
                        s[sp][t][3] = fmaf(z[3], k1[b], s[sp][t][3]);
                    }
                }
            }

            // ---- softmax: scores in units of log 2, the running maximum of each column
            const bool masked = mask != 0xffffffffu || t0 + 32 > lim_min;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int sp = 0; sp < 2; ++sp)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[sp][t][i] *= cs[t][i & 1];
                if (masked) {
#pragma unroll
                    for (int sp = 0; sp < 2; ++sp)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = 16 * sp + 8 * (i >> 1) + g;
                            if (!((mask >> row) & 1) || t0 + row >= lim[t][i & 1]) s[sp][t][i] = -INFINITY;
                        }
                }
                float mx[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) mx[i] = fmaxf(fmaxf(s[0][t][i], s[0][t][2 + i]), fmaxf(s[1][t][i], s[1][t][2 + i]));
                if (__any_sync(0xffffffffu, mx[0] > m[t][0] || mx[1] > m[t][1])) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v = mx[i];
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        const float al = v > m[t][i] ? ex2(m[t][i] - v) : 1.0f;
                        m[t][i] = fmaxf(m[t][i], v);
                        l[t][i] *= al;
#pragma unroll
                        for (int k = 0; k < MT; ++k) {
                            o[t][k][i] *= al;
                            o[t][k][2 + i] *= al;
                        }
                    }
                }
                // a column that has seen nothing has maximum -infinity: its probabilities are zeros
                // (2^15 of each: the sum has the factor, too)
                const float mu[2] = {m[t][0] == -INFINITY ? 0.0f : m[t][0] - 15.0f, m[t][1] == -INFINITY ? 0.0f : m[t][1] - 15.0f};
#pragma unroll
                for (int sp = 0; sp < 2; ++sp)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[sp][t][i] = ex2(s[sp][t][i] - mu[i & 1]);
                        l[t][i & 1] += s[sp][t][i];
                    }
            }

            // ---- O^T: positions 2 c, + 1 and + 8, + 9 of a strip; channels 32 b + 4 g ..
            const uint32_t vst = ring_s + (it % ST) * C::kStage + C::kBytes + vrow * C::kRow;
            // registers: block b2's positions 2 c and 2 c + 8, then block b2 + 1's
            auto codes = [&](uint32_t (&r)[4], int sp, int b2) {
                ldmatrix_trans(r, vst + 16 * sp * C::kRow + ((min(b2 + vsel, NB - 1) ^ vsw) << 4));
            };
            auto factors = [&](uint32_t (&f)[4], int pair) {
                const uint4 v = *reinterpret_cast<const uint4 *>(vtab + pair * 4);
                f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
            };
            if (!wide) {
#pragma unroll
                for (int sp = 0; sp < 2; ++sp) {
                    uint32_t f0[4], f1[4], pt[NT][2];
                    factors(f0, 8 * sp + c);
                    factors(f1, 8 * sp + 4 + c);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        pt[t][0] = movmatrix(gemv::pack_f16x2(s[sp][t][0], s[sp][t][1]));
                        pt[t][1] = movmatrix(gemv::pack_f16x2(s[sp][t][2], s[sp][t][3]));
                    }
#pragma unroll
                    for (int b2 = 0; b2 < NB; b2 += 2) {
                        uint32_t r[4];
                        codes(r, sp, b2);
#pragma unroll
                        for (int b = b2; b < b2 + 2 && b < NB; ++b) {
                            const uint32_t x = r[2 * (b - b2)], y = r[2 * (b - b2) + 1];
                            const uint32_t u = __byte_perm(x, y, 0x5410), v = __byte_perm(x, y, 0x7632);
                            uint32_t ev[4], od[4];           // codes 0, 2 (1, 3) of 2 c, + 1, then of 2 c + 8, + 9
                            gemv::codes_f16((u & 0x0F0F0F0Fu) | ((v << 4) & 0xF0F0F0F0u), ev);
                            gemv::codes_f16(((u >> 4) & 0x0F0F0F0Fu) | (v & 0xF0F0F0F0u), od);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const uint32_t p0 = hmul2_f16(pt[t][0], f0[b]), p1 = hmul2_f16(pt[t][1], f1[b]);
                                gemv::mma_f16(o[t][2 * b], ev[0], od[0], ev[2], od[2], p0, p1);
                                gemv::mma_f16(o[t][2 * b + 1], ev[1], od[1], ev[3], od[3], p0, p1);
                            }
                        }
                    }
                }
            } else {
#pragma unroll
                for (int sp = 0; sp < 2; ++sp) {
                    uint32_t f0[4], f1[4], pt[NT][2];
                    factors(f0, 8 * sp + c);
                    factors(f1, 8 * sp + 4 + c);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        pt[t][0] = movmatrix(mma::pack_bf16x2(s[sp][t][0], s[sp][t][1]));
                        pt[t][1] = movmatrix(mma::pack_bf16x2(s[sp][t][2], s[sp][t][3]));
                    }
#pragma unroll
                    for (int b2 = 0; b2 < NB; b2 += 2) {
                        uint32_t r[4];
                        codes(r, sp, b2);
#pragma unroll
                        for (int b = b2; b < b2 + 2 && b < NB; ++b) {
                            const uint32_t x = r[2 * (b - b2)], y = r[2 * (b - b2) + 1];
                            const uint32_t x0 = hmul2_bf16(code_bf16<0>(x), f0[b]), x1 = hmul2_bf16(code_bf16<1>(x), f0[b]);
                            const uint32_t x2 = hmul2_bf16(code_bf16<2>(x), f0[b]), x3 = hmul2_bf16(code_bf16<3>(x), f0[b]);
                            const uint32_t y0 = hmul2_bf16(code_bf16<0>(y), f1[b]), y1 = hmul2_bf16(code_bf16<1>(y), f1[b]);
                            const uint32_t y2 = hmul2_bf16(code_bf16<2>(y), f1[b]), y3 = hmul2_bf16(code_bf16<3>(y), f1[b]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                mma_bf16(o[t][2 * b], x0, x1, y0, y1, pt[t][0], pt[t][1]);
                                mma_bf16(o[t][2 * b + 1], x2, x3, y2, y3, pt[t][0], pt[t][1]);
                            }
                        }
                    }
                }
            }
        }
        gemv::cp_wait<0>();

        // ---- the warps' results together: output [W][R][D], maxima and sums [W][R].  Outputs stay relative to the
        // largest value scale until they are divided by the sum: 2^15 times a sum of many of the largest values is
        // past fp32.
        if (lane == 0) vtops[warp] = vtop;
        __syncthreads();
        float *ow = reinterpret_cast<float *>(smem_few), *mw = ow + W * R * C::kOutRow, *lw = mw + W * R;
        int vmax = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) vmax = max(vmax, vtops[w]);
        const float vs = pow2(vtop - vmax), vscale = pow2(vmax - 126);       // (half of it is in `inv`)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = l[t][i];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                const int r = 8 * t + 2 * c + i;
                if (g == 0) {
                    mw[warp * R + r] = m[t][i];
                    lw[warp * R + r] = v;
                }
                float *dst = ow + (warp * R + r) * C::kOutRow + 4 * g;
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    *reinterpret_cast<float4 *>(dst + 32 * b) =
                        make_float4(o[t][2 * b][i] * vs, o[t][2 * b][2 + i] * vs, o[t][2 * b + 1][i] * vs, o[t][2 * b + 1][2 + i] * vs);
            }
        __syncthreads();
        const bool whole = count == units;
        float *sl = nullptr;
        if (!whole) sl = slot<R, D>(a, 2 * blockIdx.x + (p.unit == 0 ? 1 : 0));
        for (int i = threadIdx.x; i < R * D / 2; i += W * 32) {
            const int r = i / (D / 2), d = 2 * (i % (D / 2)), row = r0 + r;
            if (row >= q.rows) break;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < W; ++w) mm = fmaxf(mm, mw[w * R + r]);
            float ll = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float mwr = mw[w * R + r], lwr = lw[w * R + r];
                // a warp that saw nothing has nothing; a NaN score makes its sum NaN and reaches the result
                const float f = mwr == -INFINITY ? (lwr == 0.0f ? 0.0f : lwr) : ex2(mwr - mm);
                ll = fmaf(lwr, f, ll);
                const float2 v = *reinterpret_cast<const float2 *>(ow + (w * R + r) * C::kOutRow + d);
                x = fmaf(v.x, f, x);
                y = fmaf(v.y, f, y);
            }
            float inv = 0.5f / ll;
            if (ll == 0.0f) inv = whole ? empty_row(a, p.b, row_end(a, q, row)) : 0.0f;
            x = x * inv * vscale;
            y = y * inv * vscale;
            if (nan_first[d / 32] < row_end(a, q, row)) x = y = __uint_as_float(0x7fc00000u);
            if (whole) {
                *reinterpret_cast<uint32_t *>(a.out + (int64_t(q.lo + row / a.group) * a.hq + p.h * a.group + row % a.group) * D +
                                              d) = mma::pack_bf16x2(x, y);
            } else {
                *reinterpret_cast<float2 *>(sl + slot_at<R>(r, d)) = make_float2(x, y);
                if (d == 0) {
                    sl[R * D + r] = mm;
                    sl[R * D + R + r] = ll;
                }
            }
        }
        if (!whole && p.unit == 0 && threadIdx.x == 0) {
            // the item starts here and goes on: the shares up to the one with its last unit hold it
            const int64_t last = quotient(total * (blockIdx.x + 1), shares) - left + units - 1;
            *desc = Desc{int(share_of(last, total, shares)) - int(blockIdx.x) + 1, p.h, r0, q.lo, q.rows, p.b, {}};
        }
        __syncthreads();
        left -= count + C::kItemCost;
        if (left > 0) next_item<R>(a, q, p);
    }
}

// The items that were split: the CTAs of share i (R / ROWS, ROWS rows each) add
// up the partials of the item that began in its slot 2 i + 1 and went on in
// slots 2 (i + 1), 2 (i + 2), ...
template <int R, int D, int THREADS, int ROWS>
__global__ void __launch_bounds__(THREADS)
merge_kernel(const Args a)
{
    pdl_wait();
    __shared__ float weight[ROWS][kMaxCtas];                   // of each part: its share of the sum
    const int share = int(blockIdx.x) / (R / ROWS), first = int(blockIdx.x) % (R / ROWS) * ROWS;
    const Desc d = reinterpret_cast<const Desc *>(a.work)[share];
    if (d.parts == 0) return;
    const int r0 = d.r0 + first, rows = min(ROWS, d.rows - r0);
    if (rows <= 0) return;
    auto part = [&](int k) { return slot<R, D>(a, k ? 2 * (share + k) : 2 * share + 1); };
    // four channels of a row per thread, the parts dealt out to G groups of threads where there are more threads;
    // the first two parts are on their way while the weights are found
    constexpr int E = ROWS * D / 4, G = THREADS / E;
    static_assert(G >= 1, "a thread for every four channels");
    __shared__ float4 some[G][E];
    const int e = threadIdx.x % E, grp = threadIdx.x / E, er = e % ROWS, ech = 4 * (e / ROWS);
    const bool mine = grp < G && er < rows;
    auto values = [&](int k) {
        return mine && k < d.parts ? *reinterpret_cast<const float4 *>(part(k) + slot_at<R>(first + er, ech))
                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    const float4 v0 = values(grp), v1 = values(grp + G);
    // a warp per row: the maximum, then every part's weight and the sum, lanes over the parts
    for (int r = threadIdx.x / 32; r < rows; r += THREADS / 32) {
        const int lane = threadIdx.x % 32;
        float mm = -INFINITY, lk_first = 0.0f;
        for (int k = lane; k < d.parts; k += 32) {
            const float mk = part(k)[R * D + first + r];
            lk_first = k == lane ? part(k)[R * D + R + first + r] : lk_first;
            weight[r][k] = mk;
            mm = fmaxf(mm, mk);
        }
#pragma unroll
        for (int i = 16; i; i >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, i));
        float ll = 0.0f;
        for (int k = lane; k < d.parts; k += 32) {
            const float mk = weight[r][k], lk = k == lane ? lk_first : part(k)[R * D + R + first + r];
            // a part that saw nothing has nothing; a NaN sum reaches the result
            const float f = mk == -INFINITY ? (lk == 0.0f ? 0.0f : lk) : lk * ex2(mk - mm);
            weight[r][k] = f;
            ll += f;
        }
#pragma unroll
        for (int i = 16; i; i >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, i);
        const float inv = ll == 0.0f ? empty_row(a, d.b, row_end(a, load_seq(a, d.b), r0 + r)) : 1.0f / ll;
        for (int k = lane; k < d.parts; k += 32) weight[r][k] *= inv;
    }
    __syncthreads();
    if (mine) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        auto add = [&](const float4 v, float f) {
            x.x = fmaf(v.x, f, x.x);
            x.y = fmaf(v.y, f, x.y);
            x.z = fmaf(v.z, f, x.z);
            x.w = fmaf(v.w, f, x.w);
        };
        if (grp < d.parts) add(v0, weight[er][grp]);
        if (grp + G < d.parts) add(v1, weight[er][grp + G]);
#pragma unroll 8
        for (int k = grp + 2 * G; k < d.parts; k += G) add(values(k), weight[er][k]);
        some[grp][e] = x;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * D / 4; i += THREADS) {              // by rows for the output
        const int r = i / (D / 4), ch = i % (D / 4), row = r0 + r;
        float4 x = some[0][ch * ROWS + r];
#pragma unroll
        for (int k = 1; k < G; ++k) {
            const float4 v = some[k][ch * ROWS + r];
            x.x += v.x;
            x.y += v.y;
            x.z += v.z;
            x.w += v.w;
        }
        *reinterpret_cast<uint2 *>(a.out + (int64_t(d.lo + row / a.group) * a.hq + d.h * a.group + row % a.group) * D + 4 * ch) =
            make_uint2(mma::pack_bf16x2(x.x, x.y), mma::pack_bf16x2(x.z, x.w));
    }
}

}  // namespace attn
