// mx_attention.cuh -- attention of a chunk of new tokens over a paged MXFP4
// cache.  Included by kroquant.cu; uses its helpers, mx_cache.cuh and
// mxf4_gemv.cuh.
//
//   out[t][h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[t][h] . k_j - max)
//
// over the positions j of t's sequence that its mask leaves: j <= the
// position of t (causal) or every j below the sequence's length.  Positions
// whose page the table does not name are not seen.  A row that sees nothing
// is zero.
//
// Work.  The query heads of a kv head and the new tokens of a sequence are the
// rows of one product over that head's cache: row r of (sequence b, kv head h)
// is token r / g, query head h g + r % g.  An item is R consecutive rows of one
// (b, h); it takes ceil(end / 128) units of 128 positions, end being the last
// position that any of its rows sees.  The units of all items, in order, are
// dealt out in equal contiguous shares to a grid that fills the GPU once, from
// the lengths on the device: no plan on the host, ragged batches balance, and
// long sequences split over as many CTAs as they need.  A CTA whose share ends
// inside an item leaves a partial result (maximum, sum, unnormalised output)
// in its slot of the workspace, and merge_kernel adds up the partials of the
// items that were split, in order: the same lengths give the same bits.

namespace attn {

constexpr int kUnit = 128;                   // positions per unit of work
constexpr int kMaxCtas = 512;                // shares (the workspace has two slots for each)
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

// What a CTA left behind: the item that its share ended in (rows > 0: split
// there, `parts` shares hold it, this one the first).
struct Desc {
    int b, h, tile, parts;
};

// Slot i of a workspace for R rows: unnormalised output [R][D], maxima [R], sums [R].
template <int R, int D>
__device__ __forceinline__ float *slot(const Args &a, int i)
{
    return reinterpret_cast<float *>(a.work + kMaxCtas * sizeof(Desc)) + int64_t(i) * R * (D + 2);
}

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

template <int R>
__device__ __forceinline__ int64_t head_units(const Args &a, const Seq &q)
{
    const int tiles = (q.rows + R - 1) / R;
    if (!a.causal) return int64_t(tiles) * (tiles ? item_units<R>(a, q, 0) : 0);
    int64_t u = 0;
    for (int t = 0; t < tiles; ++t) u += item_units<R>(a, q, t);
    return u;
}

// A place in the order of units: sequence, head, tile, unit of the item.
struct Place {
    int b, h, tile, unit;
};

// The share of this CTA: its first unit's place and the number of units.  There
// are `shares` of them, one for each CTA but no more than units, so that every
// share between an item's first and last holds a part of it.  Every thread of
// the CTA calls it; `sh` is shared memory of 34 int64.
template <int R, int THREADS>
__device__ __forceinline__ int64_t my_share(const Args &a, int64_t *sh, Place &p, int64_t &total, int64_t &first,
                                            int &shares)
{
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int per = (a.s.B + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, a.s.B), b1 = min(b0 + per, a.s.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += head_units<R>(a, load_seq(a, b)) * a.s.heads;
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) sh[warp] = incl;
    __syncthreads();
    int64_t base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += sh[w];
        total += sh[w];
    }
    shares = int(min(int64_t(gridDim.x), total));
    if (int(blockIdx.x) >= shares) return 0;
    first = total * blockIdx.x / shares;
    const int64_t last = total * (blockIdx.x + 1) / shares;
    int64_t at = base + incl - mine;         // units before this thread's sequences
    int *place = reinterpret_cast<int *>(sh + 32);
    if (first >= at && first < at + mine) {
        int b = b0;
        Seq q;
        int64_t hu;
        for (;; ++b) {                       // ends: the units of b0 .. b1 - 1 hold `first`
            q = load_seq(a, b);
            hu = head_units<R>(a, q);
            if (first < at + hu * a.s.heads) break;
            at += hu * a.s.heads;
        }
        int64_t off = first - at;
        const int h = int(off / hu);
        off -= h * hu;
        int t = 0;
        for (int u = item_units<R>(a, q, 0); off >= u; u = item_units<R>(a, q, ++t)) off -= u;
        place[0] = b;
        place[1] = h;
        place[2] = t;
        place[3] = int(off);
    }
    __syncthreads();
    p = Place{place[0], place[1], place[2], place[3]};
    return last - first;
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
// operand: values are expanded to bf16 by shifts (the code's bits 8, 7, 6 and
// 15 are code * 2^-126, which one packed multiply by 2^(126 + scale) makes
// exact: fp32's range in 8 bits), relative to the warp's running largest value
// scale, with P in bf16: half a step, 2^-8 of each probability.
// P^T leaves the first product with positions along the rows and enters the
// second along the columns: movmatrix transposes it.
//
// A CTA is four warps, each with its own softmax state and its own cp.async
// ring of stages (32 positions of keys, values and scales); a warp takes every
// fourth stage of the share and waits for nothing but its own copies.  They
// meet when an item ends.
template <int D_, int NT_>
struct Few {
    static constexpr int D = D_, NT = NT_;
    static constexpr int R = 8 * NT;
    static constexpr int kWarps = 4;
    static constexpr int kStages = 3;
    static constexpr int NB = D / 32;
    static constexpr int DP = D <= 64 ? 64 : 128;            // channels of the V tile (D = 32, 96: the rest is not stored)
    static constexpr int MT = DP / 16;
    static constexpr int kKRow = D >= 96 ? 64 : D / 2;       // bytes of a key's row in the stage
    static constexpr int kVRow = DP / 2;
    static constexpr int kKBytes = 32 * kKRow, kVBytes = 32 * kVRow;
    static constexpr int kScaleBytes = 32 * NB;              // of keys; the values' follow
    static constexpr int kStage = kKBytes + kVBytes + 2 * kScaleBytes;
    static constexpr int kTable = 32 * 4 * 4 + 16 * 4 * 4;   // key scales (fp32), value scales (bf16 pairs)
    static constexpr int kWarpBytes = kStages * kStage + kTable;
    static constexpr int kOutRow = D + 4;                    // floats
    static constexpr int kMerge = kWarps * R * (kOutRow + 2) * 4;
    static constexpr int kSmem = kWarps * kWarpBytes > kMerge ? kWarps * kWarpBytes : kMerge;
};

__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

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
    extern __shared__ __align__(16) uint8_t smem_dyn[];
    __shared__ int64_t sh[34];
    __shared__ int nan_first[4];             // per 32 channels: the first position of the item whose value is NaN
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;

    Place p;
    int64_t total, first;
    int shares;
    int64_t left = my_share<R, W * 32>(a, sh, p, total, first, shares);
    Desc *desc = reinterpret_cast<Desc *>(a.work) + blockIdx.x;
    if (threadIdx.x == 0) *desc = Desc{0, 0, 0, 0};
    if (left <= 0) return;
    int64_t at_unit = first;                 // among all units

    uint8_t *ring = smem_dyn + warp * C::kWarpBytes;
    float *ktab = reinterpret_cast<float *>(ring + ST * C::kStage);          // [32 positions][4]
    uint32_t *vtab = reinterpret_cast<uint32_t *>(ktab + 128);               // [16 pairs][4]
    const uint32_t ring_s = smem_addr(ring);
    const int vblk = C::DP == 128 ? g >> 1 : g >> 2;         // the 32 channels that this thread's V rows are in

    Seq q = load_seq(a, p.b);
    while (left > 0) {
        // ---- the segment: units [p.unit, p.unit + count) of item (b, h, tile)
        const int units = item_units<R>(a, q, p.tile);
        const int count = int(min(left, int64_t(units - p.unit)));
        const int r0 = p.tile * R;
        const int item_end = row_end(a, q, min(r0 + R, q.rows) - 1);
        const int t_end = min(item_end, (p.unit + count) * kUnit);
        const int32_t *table = a.s.table + int64_t(p.b) * a.s.table_stride;

        // q as the 8-column operand: fp16, a power of two per row
        uint32_t qf[NT][NB][4];
        int qexp[NT];                                        // of row 8 nt + g
        int lim[NT][2], lim_min = 0x7fffffff;                // of rows 8 nt + 2 c, + 1
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = r0 + 8 * t + g;
            uint4 raw[NB];
            uint32_t top = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                raw[b] = make_uint4(0u, 0u, 0u, 0u);
                if (r < q.rows)
                    raw[b] = __ldg(reinterpret_cast<const uint4 *>(a.q + int64_t(q.lo + r / a.group) * a.q_st +
                                                                   int64_t(p.h * a.group + r % a.group) * a.q_sh +
                                                                   32 * b + 8 * c));
                const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
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
                const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
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
        int vtop = 0;                                        // the largest value scale byte so far
        uint32_t on_page = 0;                                // two bits per stage in flight: its strips have a page

        const int t_first = p.unit * kUnit + warp * 32;
        auto fetch = [&](int t0, int slot_i) {               // stage: positions t0 .. t0 + 31
            uint32_t bits = 0;
            if (t0 < t_end) {
                int64_t row[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    row[s] = t0 + 16 * s < t_end ? strip_row(a, table, p.h, t0 + 16 * s) : -1;
                    bits |= row[s] >= 0 ? 1u << s : 0u;
                }
                const uint32_t dst = ring_s + slot_i * C::kStage;
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const int idx = lane + 32 * j, s = idx / (16 * NB), in = idx - s * 16 * NB;
                    const int r = in / NB, ch = in % NB;
                    const int64_t rw = s ? row[1] : row[0];
                    const uint32_t size = rw >= 0 ? 16 : 0;
                    const int64_t off = (rw >= 0 ? rw : 0) * (D / 2) + in * 16;
                    const int kch = D >= 96 ? ch ^ ((r >> 1) & 3) : D == 64 ? ch ^ ((r >> 2) & 1) : ch;
                    gemv::cp_async16_sized(dst + (16 * s + r) * C::kKRow + kch * 16, size ? a.kc + off : a.kc, size);
                    const int vs = (r & 8) | ((r & 1) << 2) | ((r >> 1) & 3);
                    const int vch = C::DP == 128 ? ch ^ (vs & 2) : ch;
                    gemv::cp_async16_sized(dst + C::kKBytes + (16 * s + vs) * C::kVRow + vch * 16, size ? a.vc + off : a.vc,
                                           size);
                }
                if (lane < 4 * NB) {                         // scales: 16 NB bytes of a strip are contiguous
                    const int s = (lane / NB) & 1, piece = lane % NB;
                    const bool is_v = lane >= 2 * NB;
                    const int64_t rw = s ? row[1] : row[0];
                    const uint8_t *base = is_v ? a.vs : a.ks;
                    gemv::cp_async16_sized(dst + C::kKBytes + C::kVBytes + lane * 16,
                                           rw >= 0 ? base + rw * NB + piece * 16 : base, rw >= 0 ? 16 : 0);
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
            int kb[NB], vb[NB], ktop = 0, vmax = 0;
            bool vnan = false;
            {
                const uint8_t *ks = st + C::kKBytes + C::kVBytes + lane * NB;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    kb[b] = ks[b];
                    vb[b] = valid ? ks[C::kScaleBytes + b] : 0;
                    if (kb[b] < int(kNanByte)) ktop = max(ktop, valid ? kb[b] : 0);
                    if (vb[b] >= int(kNanByte)) vnan = true;
                    else vmax = max(vmax, vb[b]);
                }
            }
            if (__any_sync(0xffffffffu, vnan)) {             // rare: values that are NaN count as zero here
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    if (vb[b] >= int(kNanByte)) {
                        atomicMin(&nan_first[b], t0 + lane);
                        vb[b] = -1;
                    }
            }
            ktop = __reduce_max_sync(0xffffffffu, ktop);
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
            {
                float kv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    kv[b] = kb[b] >= int(kNanByte) ? __uint_as_float(0x7fc00000u) : pow2(kb[b] - ktop);
                    // bf16 2^(126 + byte - vtop): at most 2^126, zero for a position that counts for nothing
                    const uint32_t f = valid && vb[b] >= 0 ? uint32_t(max(vb[b] - vtop + 253, 0)) << 7 : 0u;
                    reinterpret_cast<uint16_t *>(vtab)[((lane >> 1) * 4 + b) * 2 + (lane & 1)] = uint16_t(f);
                }
                *reinterpret_cast<float4 *>(ktab + 4 * lane) = make_float4(kv[0], kv[1], kv[2], kv[3]);
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
                    const uint8_t *kr = st + (16 * sp + g) * C::kKRow + ch * 16 + 4 * c;
                    uint32_t x[4], y[4];
                    gemv::codes_f16(*reinterpret_cast<const uint32_t *>(kr), x);
                    gemv::codes_f16(*reinterpret_cast<const uint32_t *>(kr + 8 * C::kKRow), y);
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
            uint32_t pt[2][NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float mx[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float cs = a.scale_log2 * pow2(max(min(qe[t][i] + ktop - 127, 127), -126));
#pragma unroll
                    for (int sp = 0; sp < 2; ++sp) {
                        s[sp][t][i] *= cs;
                        s[sp][t][2 + i] *= cs;
                    }
                    if (masked) {
#pragma unroll
                        for (int sp = 0; sp < 2; ++sp)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const int row = 16 * sp + 8 * hf + g;
                                if (!((mask >> row) & 1) || t0 + row >= lim[t][i]) s[sp][t][2 * hf + i] = -INFINITY;
                            }
                    }
                    float v = fmaxf(fmaxf(s[0][t][i], s[0][t][2 + i]), fmaxf(s[1][t][i], s[1][t][2 + i]));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    mx[i] = fmaxf(m[t][i], v);
                }
                if (__any_sync(0xffffffffu, mx[0] > m[t][0] || mx[1] > m[t][1])) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float al = mx[i] > m[t][i] ? ex2(m[t][i] - mx[i]) : 1.0f;
                        m[t][i] = mx[i];
                        l[t][i] *= al;
#pragma unroll
                        for (int k = 0; k < MT; ++k) {
                            o[t][k][i] *= al;
                            o[t][k][2 + i] *= al;
                        }
                    }
                }
                // a column that has seen nothing has maximum -infinity: its probabilities are zeros
                const float mu[2] = {m[t][0] == -INFINITY ? 0.0f : m[t][0], m[t][1] == -INFINITY ? 0.0f : m[t][1]};
#pragma unroll
                for (int sp = 0; sp < 2; ++sp) {
                    float e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e[i] = ex2(s[sp][t][i] - mu[i & 1]);
                        l[t][i & 1] += e[i];
                    }
                    pt[sp][t][0] = movmatrix(mma::pack_bf16x2(e[0], e[1]));
                    pt[sp][t][1] = movmatrix(mma::pack_bf16x2(e[2], e[3]));
                }
            }

            // ---- O^T: positions 2 c, + 1 and + 8, + 9 of a strip; channels DP / 8 * g ..
#pragma unroll
            for (int sp = 0; sp < 2; ++sp) {
                const uint32_t fa = vtab[(8 * sp + c) * 4 + vblk], fb = vtab[(8 * sp + 4 + c) * 4 + vblk];
                const uint8_t *vr = st + C::kKBytes + (16 * sp + c) * C::kVRow;
                constexpr int WPT = C::DP / 64;              // words of a position per thread
                uint32_t w[4][WPT];                          // positions 2 c, 2 c + 1, 2 c + 8, 2 c + 9: slots c, + 4, + 8, + 12
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (C::DP == 128) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(vr + 4 * k * C::kVRow + (((g >> 1) ^ (c & 2)) << 4) +
                                                                         (g & 1) * 8);
                        w[k][0] = v.x;
                        w[k][1] = v.y;
                    } else {
                        w[k][0] = *reinterpret_cast<const uint32_t *>(vr + 4 * k * C::kVRow + 4 * g);
                    }
                }
#pragma unroll
                for (int x = 0; x < WPT; ++x)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {         // four codes of both positions
                        const uint32_t sel = hf ? 0x7632 : 0x5410;
                        const uint32_t u = __byte_perm(w[0][x], w[1][x], sel), v = __byte_perm(w[2][x], w[3][x], sel);
                        const uint32_t a0 = hmul2_bf16(code_bf16<0>(u), fa), a1 = hmul2_bf16(code_bf16<1>(u), fa);
                        const uint32_t a2 = hmul2_bf16(code_bf16<2>(u), fa), a3 = hmul2_bf16(code_bf16<3>(u), fa);
                        const uint32_t b0 = hmul2_bf16(code_bf16<0>(v), fb), b1 = hmul2_bf16(code_bf16<1>(v), fb);
                        const uint32_t b2 = hmul2_bf16(code_bf16<2>(v), fb), b3 = hmul2_bf16(code_bf16<3>(v), fb);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            mma_bf16(o[t][4 * x + 2 * hf], a0, a1, b0, b1, pt[sp][t][0], pt[sp][t][1]);
                            mma_bf16(o[t][4 * x + 2 * hf + 1], a2, a3, b2, b3, pt[sp][t][0], pt[sp][t][1]);
                        }
                    }
            }
        }
        gemv::cp_wait<0>();

        // ---- the warps' results together: output [W][R][D], maxima and sums [W][R]
        __syncthreads();
        float *ow = reinterpret_cast<float *>(smem_dyn), *mw = ow + W * R * C::kOutRow, *lw = mw + W * R;
        const float vs = pow2(vtop - 127);
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
                float *dst = ow + (warp * R + r) * C::kOutRow + g * (C::DP / 8);
#pragma unroll
                for (int k = 0; k < MT; ++k)
                    if (g * (C::DP / 8) + 2 * k < D)
                        *reinterpret_cast<float2 *>(dst + 2 * k) = make_float2(o[t][k][i] * vs, o[t][k][2 + i] * vs);
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
            if (nan_first[d / 32] < row_end(a, q, row)) x = y = __uint_as_float(0x7fc00000u);
            if (whole) {
                const float inv = 1.0f / ll;
                const uint32_t v = ll == 0.0f && x == 0.0f ? 0u : mma::pack_bf16x2(x * inv, y * inv);
                *reinterpret_cast<uint32_t *>(a.out + (int64_t(q.lo + row / a.group) * a.hq + p.h * a.group + row % a.group) * D +
                                              d) = v;
            } else {
                *reinterpret_cast<float2 *>(sl + r * D + d) = make_float2(x, y);
                if (d == 0) {
                    sl[R * D + r] = mm;
                    sl[R * D + R + r] = ll;
                }
            }
        }
        if (!whole && p.unit == 0 && threadIdx.x == 0) {
            // the item starts here and goes on: the shares up to the one with its last unit hold it
            const int64_t last = at_unit + units - 1;
            int64_t k = blockIdx.x + 1;
            while (total * (k + 1) / shares <= last) ++k;
            *desc = Desc{p.b, p.h, p.tile, int(k - blockIdx.x + 1)};
        }
        __syncthreads();
        at_unit += count;
        left -= count;
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
    const int share = int(blockIdx.x) / (R / ROWS), first = int(blockIdx.x) % (R / ROWS) * ROWS;
    const Desc d = reinterpret_cast<const Desc *>(a.work)[share];
    if (d.parts == 0) return;
    const Seq q = load_seq(a, d.b);
    const int r0 = d.tile * R;
    for (int i = threadIdx.x; i < ROWS * D / 2; i += THREADS) {
        const int r = first + i / (D / 2), ch = 2 * (i % (D / 2)), row = r0 + r;
        if (row >= q.rows) break;
        float mm = -INFINITY, ll = 0.0f, x = 0.0f, y = 0.0f;
        for (int k = 0; k < d.parts; ++k) {
            const float *sl = slot<R, D>(a, k ? 2 * (share + k) : 2 * share + 1);
            const float mk = sl[R * D + r], lk = sl[R * D + R + r];
            const float2 v = *reinterpret_cast<const float2 *>(sl + r * D + ch);
            const float mn = fmaxf(mm, mk);
            const float f0 = mm == -INFINITY ? 0.0f : ex2(mm - mn);
            const float f1 = mk == -INFINITY ? (lk == 0.0f ? 0.0f : lk) : ex2(mk - mn);
            // (0 * NaN: what an earlier part made NaN stays so)
            x = fmaf(v.x, f1, mm == -INFINITY && x == x ? 0.0f : x * f0);
            y = fmaf(v.y, f1, mm == -INFINITY && y == y ? 0.0f : y * f0);
            ll = fmaf(lk, f1, mm == -INFINITY && ll == ll ? 0.0f : ll * f0);
            mm = mn;
        }
        const float inv = 1.0f / ll;
        const uint32_t v = ll == 0.0f && x == 0.0f ? 0u : mma::pack_bf16x2(x * inv, y * inv);
        *reinterpret_cast<uint32_t *>(a.out + (int64_t(q.lo + row / a.group) * a.hq + d.h * a.group + row % a.group) * D + ch) = v;
    }
}

}  // namespace attn
