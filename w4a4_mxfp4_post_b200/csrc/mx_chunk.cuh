// mx_chunk.cuh -- attention over the paged MXFP4 cache for many rows per kv
// head (chunks of prompts).  Included by kroquant.cu after mx_attention.cuh,
// whose division of the work it shares.
//
// An item is 256 consecutive rows of one (sequence, kv head): two tiles of 128
// rows.  For every unit of 128 positions the fifth-generation tensor cores
// compute, for each tile,
//   S = Q K^T   (128 x 128, over the channels)       into tensor memory
//   O += P V    (128 x channels, over the positions) P from tensor memory
// with bf16 operands and fp32 sums, P = exp2(S c - m c).
//
// Bound: 4 D flops per row and position on the tensor cores, and 16 exponentials
// per clock and SM: for D = 128 both take 1024 clocks per tile and unit.  Two
// tiles per CTA keep both busy: while one tile's softmax runs, the tensor cores
// work for the other.
//
// Keys and values are decoded to bf16 once per unit and used for 256 rows.
// code * 2^(byte - 127) is exact in bf16 for every scale byte below 253.  Of a
// word's 8 codes, one AND, one multiply by 2^12 + 2^6 and one AND put codes n
// and n + 4 side by side as bf16 numbers code * 2^-126 (code 1, 0.5, is a
// subnormal), which one packed multiply by 2^(byte - 1) makes right.  Pairs come
// out as (0,4) (1,5) (2,6) (3,7), so the channels of every group of 8 are kept
// in that order: in K and in Q (the sum does not care) and in V, whose columns
// are put back when the result is written.
//
// Roles (16 warps):
//   0-3, 4-7  softmax of tile 0, 1: a thread owns a row, so the maximum and the
//             sum need no exchange.  P overwrites the upper half of S's columns.
//             O is rescaled only when a row's maximum has grown by more than 2^8
//             since the last time (exact: P and the sum use the same stale
//             maximum, and P <= 2^8 loses nothing in bf16).
//   8-14      decode: a unit is 8 tasks, 32 positions of its keys or values each
//             (a lane per position), which the 7 warps take in turn
//   15        issues the MMAs: P0 V, Q0 K', P1 V, Q1 K' (K' the next unit's)
// Q, K and V lie in the 128-byte swizzle, 64 channels to a row of 128 bytes; K
// and Q are read K-major, V with its channels as the major dimension.
// Every wait is bounded (g_wait_timeouts).

namespace attn {
namespace chunk {

constexpr int kTile = 128;                                   // rows of a tile, positions of a unit
constexpr int R = 2 * kTile;                                 // rows of an item
constexpr int kThreads = 16 * 32;
constexpr int kDecodeWarps = 7;
constexpr int kSegs = 8;                                     // segments whose NaN positions are kept
constexpr int kRing = 2;                                     // stages of K and of V
constexpr int kMergeRows = 16;                               // rows that a CTA of the merge takes
constexpr int kMaxCtas = 192;                                // shares
constexpr float kSlack = 8.0f;                               // log2 of how far a maximum may be stale
constexpr uint32_t kO = 256;                                 // tensor memory: S of tile i at 128 i, O at 256 + 128 i
static_assert(kTile == kUnit, "a unit is a tile of positions");

template <int D_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr int NB = D / 32;
    static constexpr int kHalves = D > 64 ? 2 : 1;
    static constexpr int kTileBytes = kHalves * kTile * 128; // a tile of Q, K or V
    static constexpr int kNumBars = 4 * kRing + 10;
    static constexpr int kSmem = (2 + 2 * kRing) * kTileBytes + 1024 + kNumBars * 8;
    // kind::f16: fp32 sums, bf16 operands; S: N = 128, both K-major; O: N = D, B (bit 16) major in N
    static constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kTile >> 3) << 17) | (8u << 24);
    static constexpr uint32_t kIdescO = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (uint32_t(D >> 3) << 17) | (8u << 24);
};

// Descriptor of an operand in the 128-byte swizzle: 8-row groups 1024 bytes
// apart; `lbo` is the distance of 64-element columns of an N-major operand.
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lbo)
{
    return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (mma::kLayoutSw128 << 61);
}

// One elected lane of the warp issues (warp-uniform operands).
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p, e;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(id),
                 "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p, e;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(id),
                 "r"(accumulate)
                 : "memory");
}

// 16 columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 64 columns, waited for.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&lo)[32], float (&hi)[32])
{
    mma::tmem_ld32_nowait(taddr, lo);
    mma::tmem_ld32_nowait(taddr + 32, hi);
    tmem_wait_ld();
}

// Whole-warp wait on a barrier; false after the budget.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, long long budget)
{
    if (gemm::warp_wait(bar, parity, budget)) return true;
    if (threadIdx.x % 32 == 0) atomicAdd(&g_wait_timeouts, 1);
    return false;
}

// A position's codes and scale bytes of one array.
template <int NB>
struct Piece {
    uint4 c[NB];
    uint32_t s;                              // scale bytes
    bool on;                                 // within the segment and on a page
};

template <int NB>
__device__ __forceinline__ void load_piece(Piece<NB> &p, const uint8_t *__restrict__ codes,
                                           const uint8_t *__restrict__ scales, int64_t row)
{
    p.on = row >= 0;
    p.s = 0;
    if (!p.on) {
#pragma unroll
        for (int b = 0; b < NB; ++b) p.c[b] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const uint4 *src = reinterpret_cast<const uint4 *>(codes) + row * NB;
#pragma unroll
    for (int b = 0; b < NB; ++b) p.c[b] = __ldg(src + b);
    if constexpr (NB == 4) {
        p.s = __ldg(reinterpret_cast<const uint32_t *>(scales) + row);
    } else if constexpr (NB == 2) {
        p.s = __ldg(reinterpret_cast<const uint16_t *>(scales) + row);
    } else {
#pragma unroll
        for (int b = 0; b < NB; ++b) p.s |= uint32_t(__ldg(scales + row * NB + b)) << (8 * b);
    }
}

// Eight codes to bf16 pairs (0,4) (1,5) (2,6) (3,7), times f.
__device__ __forceinline__ uint4 decode8(uint32_t w, uint32_t f)
{
    constexpr uint32_t kA = (1u << 12) + (1u << 6), kB = (1u << 8) + (1u << 2), kM = 0x81C081C0u;
    const uint32_t v = w >> 8;
    return make_uint4(hmul2_bf16(((w & 0x000F000Fu) * kA) & kM, f), hmul2_bf16(((w & 0x00F000F0u) * kB) & kM, f),
                      hmul2_bf16(((v & 0x000F000Fu) * kA) & kM, f), hmul2_bf16(((v & 0x00F000F0u) * kB) & kM, f));
}

// A position into row `row` of the tile at `dst`.  NaN blocks become `nan`:
// NaN for keys, zeros for values, whose NaN is put into the result.
template <int NB>
__device__ __forceinline__ void decode_row(const Piece<NB> &p, uint8_t *dst, int row, uint32_t nan)
{
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint32_t s = (p.s >> (8 * b)) & 0xffu;
        // 2^(s - 1) as far as bf16 goes, for the scales above (rare) a second factor
        uint32_t f = (min(s, 128u) + 126u) << 7;
        f |= f << 16;
        const uint32_t w[4] = {p.c[b].x, p.c[b].y, p.c[b].z, p.c[b].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 v = decode8(w[i], f);
            if (s > 128u) {
                uint32_t f2 = (s - 1u) << 7;
                f2 |= f2 << 16;
                if (s >= kNanByte) {
                    v.x = v.y = v.z = v.w = nan;
                } else {
                    v.x = hmul2_bf16(v.x, f2);
                    v.y = hmul2_bf16(v.y, f2);
                    v.z = hmul2_bf16(v.z, f2);
                    v.w = hmul2_bf16(v.w, f2);
                }
            }
            const int ch = 4 * b + i;
            *reinterpret_cast<uint4 *>(dst + (ch / 8) * (kTile * 128) + row * 128 + (((ch % 8) ^ (row & 7)) << 4)) = v;
        }
    }
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
chunk_kernel(const Args a, long long budget)
{
    pdl_wait();
    constexpr int D = C::D, NB = C::NB;
    extern __shared__ __align__(16) uint8_t smem_dyn[];
    __shared__ int64_t sh[34];
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) uint32_t visible[4][4];   // of unit u % 4: the positions that are on a page, 32 to a word
    __shared__ int nan_first[kSegs][4];      // of segment i % kSegs, per 32 channels: the first position whose value is NaN
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = base, *sK = base + 2 * C::kTileBytes, *sV = sK + kRing * C::kTileBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sV + kRing * C::kTileBytes);
    uint64_t *kfull = bars, *kempty = bars + kRing, *vfull = bars + 2 * kRing, *vempty = bars + 3 * kRing;
    uint64_t *qfull = bars + 4 * kRing;      // [2] Q of the tile in shared memory, the segment before put away
    uint64_t *sfull = qfull + 2;             // [2] S ready
    uint64_t *pfull = qfull + 4;             // [2] P ready, O in order
    uint64_t *odone = qfull + 6;             // [2] a unit's P V done
    uint64_t *segdone = qfull + 8;           // a segment's MMAs done
    uint64_t *done = qfull + 9;              // all MMAs done
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&kfull[i], 4);
            mbar_init(&kempty[i], 1);
            mbar_init(&vfull[i], 4);
            mbar_init(&vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 4);
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&odone[i], 1);
        }
        mbar_init(segdone, 1);
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    Place p;
    int64_t total, first;
    int shares;
    int64_t left = my_share<R, kThreads>(a, sh, p, total, first, shares);
    Desc *dsc = reinterpret_cast<Desc *>(a.work) + blockIdx.x;
    if (tid == 0) *dsc = Desc{0, 0, 0, 0};
    if (left <= 0) return;
    if (tid < kSegs * 4) nan_first[tid / 4][tid % 4] = 0x7fffffff;
    if (warp == 15) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    mma::tc_fence_before();
    __syncthreads();
    mma::tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // Every role walks the same segments: units [p.unit, p.unit + count) of item (b, h, tile).
    Seq q = load_seq(a, p.b);
    int seg = 0;                             // segments so far
    if (warp >= 8 && warp < 15) {
        // ---------------- keys and values into shared memory
        int k = 0;                           // units of the segments so far
        int turn = warp - 8;                 // this warp's next task, counted from the segment's first
        bool ok = true;
        while (left > 0 && ok) {
            const int units = item_units<R>(a, q, p.tile), count = int(min(left, int64_t(units - p.unit)));
            const int item_end = row_end(a, q, min((p.tile + 1) * R, q.rows) - 1);
            const int t_first = p.unit * kUnit, t_end = min(item_end, t_first + count * kUnit);
            const int32_t *table = a.s.table + int64_t(p.b) * a.s.table_stride;
            // task x: unit x / 8, values if x & 4, positions 32 (x & 3) + lane
            auto row_of = [&](int64_t x) -> int64_t {
                if (x >= int64_t(count) * 8) return -1;
                const int t = t_first + int(x >> 3) * kUnit + 32 * int(x & 3) + lane;
                if (t >= t_end) return -1;
                const int64_t r = strip_row(a, table, p.h, t & ~15);
                return r < 0 ? -1 : r + (t & 15);
            };
            auto load = [&](Piece<NB> &x, int64_t task, int64_t row) {
                const bool is_v = task & 4;
                load_piece<NB>(x, is_v ? a.vc : a.kc, is_v ? a.vs : a.ks, row);
            };
            Piece<NB> next;
            load(next, turn, row_of(turn));
            int64_t ahead = row_of(turn + kDecodeWarps);
            int64_t x = turn;
            for (; x < int64_t(count) * 8; x += kDecodeWarps) {
                const Piece<NB> cur = next;
                load(next, x + kDecodeWarps, ahead);
                ahead = row_of(x + 2 * kDecodeWarps);
                const int u = int(x >> 3), part = int(x & 3), ku = k + u, st = ku % kRing, row = 32 * part + lane;
                const bool is_v = x & 4;
                if (ku >= kRing && !wait(is_v ? &vempty[st] : &kempty[st], ((ku / kRing) - 1) & 1, budget)) {
                    ok = false;
                    break;
                }
                if (is_v) {
                    bool nan = false;
#pragma unroll
                    for (int b = 0; b < NB; ++b) nan |= ((cur.s >> (8 * b)) & 0xffu) >= kNanByte;
                    if (nan) {
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            if (((cur.s >> (8 * b)) & 0xffu) >= kNanByte)
                                atomicMin(&nan_first[seg % kSegs][b], t_first + u * kUnit + row);
                    }
                } else {
                    const uint32_t on = __ballot_sync(0xffffffffu, cur.on);
                    if (lane == 0) visible[ku & 3][part] = on;
                }
                decode_row<NB>(cur, (is_v ? sV : sK) + st * C::kTileBytes, row, is_v ? 0u : 0x7fc07fc0u);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(is_v ? &vfull[st] : &kfull[st]);
            }
            turn = int(x - int64_t(count) * 8);
            k += count;
            left -= count;
            ++seg;
            if (left > 0) next_item<R>(a, q, p);
        }
    } else if (warp == 15) {
        // ---------------- the MMAs
        int k = 0, n0 = 0, n1 = 0;           // units, units of each tile so far
        bool ok = true;
        const uint32_t aQ = smem_addr(sQ), aK = smem_addr(sK), aV = smem_addr(sV);
        auto qk = [&](int i, int st) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const uint32_t off = (j / 4) * (kTile * 128) + (j % 4) * 32;
                umma_ss(tmem + i * 128, desc(aQ + i * C::kTileBytes + off, 16), desc(aK + st * C::kTileBytes + off, 16),
                        C::kIdescS, j > 0);
            }
            gemm::umma_commit_w(&sfull[i]);
        };
        auto pv = [&](int i, int st, bool add) {
#pragma unroll
            for (int j = 0; j < kTile / 16; ++j)
                umma_ts(tmem + kO + i * 128, tmem + i * 128 + 64 + j * 8,
                        desc(aV + st * C::kTileBytes + j * 16 * 128, kTile * 128), C::kIdescO, add || j > 0);
            gemm::umma_commit_w(&odone[i]);
        };
        while (left > 0 && ok) {
            const int units = item_units<R>(a, q, p.tile), count = int(min(left, int64_t(units - p.unit)));
            const bool two = q.rows - p.tile * R > kTile;
            if (!wait(&kfull[k % kRing], (k / kRing) & 1, budget) || !wait(&qfull[0], seg & 1, budget) ||
                !wait(&qfull[1], seg & 1, budget))
                break;
            mma::tc_fence_after();
            qk(0, k % kRing);
            if (two) qk(1, k % kRing);
            gemm::umma_commit_w(&kempty[k % kRing]);
            for (int u = 0; u < count; ++u, ++k) {
                const int st = k % kRing, sn = (k + 1) % kRing;
                const bool more = u + 1 < count;
                if (!wait(&vfull[st], (k / kRing) & 1, budget) || !wait(&pfull[0], n0 & 1, budget)) {
                    ok = false;
                    break;
                }
                ++n0;
                mma::tc_fence_after();
                pv(0, st, u > 0);
                if (!two) gemm::umma_commit_w(&vempty[st]);
                if (more) {
                    if (!wait(&kfull[sn], ((k + 1) / kRing) & 1, budget)) {
                        ok = false;
                        break;
                    }
                    mma::tc_fence_after();
                    qk(0, sn);
                }
                if (two) {
                    if (!wait(&pfull[1], n1 & 1, budget)) {
                        ok = false;
                        break;
                    }
                    ++n1;
                    mma::tc_fence_after();
                    pv(1, st, u > 0);
                    gemm::umma_commit_w(&vempty[st]);
                    if (more) qk(1, sn);
                }
                if (more) gemm::umma_commit_w(&kempty[sn]);
            }
            if (!ok) break;
            gemm::umma_commit_w(segdone);
            ++seg;
            left -= count;
            if (left > 0) next_item<R>(a, q, p);
        }
        // every MMA issued has completed before the tensor memory is freed
        gemm::umma_commit_w(done);
        wait(done, 0, budget);
    } else {
        // ---------------- softmax: thread = row
        const int i = warp / 4, row = tid % kTile;
        const uint32_t lanes = uint32_t(warp % 4) << 21;                     // 32 (warp % 4) in the lane field
        const uint32_t tS = tmem + lanes + i * 128, tP = tS + 64, tO = tmem + lanes + kO + i * 128;
        int n = 0;                           // units of this tile so far
        int k = 0;                           // units so far
        const float c = a.scale_log2 == 0.0f ? 1.0f : fabsf(a.scale_log2);
        bool ok = true;
        while (left > 0 && ok) {
            const int units = item_units<R>(a, q, p.tile), count = int(min(left, int64_t(units - p.unit)));
            const int r0 = p.tile * R + i * kTile, r = r0 + row;
            // Nobody writes this segment's slot yet, and whoever read it (five segments ago) is through: the next
            // segment's first MMA waits for both tiles' softmax.
            if (tid < 4) nan_first[(seg + 3) % kSegs][tid] = 0x7fffffff;
            if (r0 >= q.rows) {
                // nothing to do, but the next segment begins after both tiles' last, and this tile's arrivals must
                // not run ahead of the segments
                __syncwarp();
                if (lane == 0) mbar_arrive(&qfull[i]);
                if (!wait(segdone, seg & 1, budget)) break;
            } else {
                const bool mine = r < q.rows;
                const int token = r / a.group, head = p.h * a.group + r - token * a.group;
                // Q: rows of the tile, channels of 8 in the decoders' order; the sign (or zero) of the scale goes into it
                {
                    const __nv_bfloat16 *src = a.q + int64_t(q.lo + token) * a.q_st + int64_t(head) * a.q_sh;
                    uint8_t *dst = sQ + i * C::kTileBytes + row * 128;
                    const uint32_t sgn = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
                    for (int ch = 0; ch < D / 8; ++ch) {
                        uint4 w = make_uint4(0u, 0u, 0u, 0u);
                        if (mine) w = __ldg(reinterpret_cast<const uint4 *>(src) + ch);
                        if (a.scale_log2 == 0.0f) {
                            w.x = hmul2_bf16(w.x, 0u);
                            w.y = hmul2_bf16(w.y, 0u);
                            w.z = hmul2_bf16(w.z, 0u);
                            w.w = hmul2_bf16(w.w, 0u);
                        }
                        *reinterpret_cast<uint4 *>(dst + (ch / 8) * (kTile * 128) + (((ch % 8) ^ (row & 7)) << 4)) =
                            make_uint4(__byte_perm(w.x, w.z, 0x5410) ^ sgn, __byte_perm(w.x, w.z, 0x7632) ^ sgn,
                                       __byte_perm(w.y, w.w, 0x5410) ^ sgn, __byte_perm(w.y, w.w, 0x7632) ^ sgn);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&qfull[i]);
                }
                const int lim = mine ? row_end(a, q, r) : 0x7fffffff;        // a row that is not there sees all, for nothing
                float m = -INFINITY, l = 0.0f;                               // m: of S, as used
                for (int u = 0; u < count; ++u, ++n) {
                    if (!wait(&sfull[i], n & 1, budget)) {
                        ok = false;
                        break;
                    }
                    mma::tc_fence_after();
                    const int t0 = (p.unit + u) * kUnit;
                    uint32_t vis[4];
                    bool masked = lim < t0 + kUnit;
                    {
                        const uint4 on = *reinterpret_cast<const uint4 *>(visible[(k + u) & 3]);
                        vis[0] = on.x, vis[1] = on.y, vis[2] = on.z, vis[3] = on.w;
                        masked |= (on.x & on.y & on.z & on.w) != 0xffffffffu;
                    }
                    masked = __any_sync(0xffffffffu, masked);
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int see = lim - t0 - 32 * j;
                            vis[j] &= see >= 32 ? 0xffffffffu : see <= 0 ? 0u : (1u << see) - 1u;
                        }
                    }
                    auto mask = [&](float (&v)[32], uint32_t bits) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = (bits >> e) & 1 ? v[e] : -INFINITY;
                    };
                    float x[32], y[32];
                    float top = m, top2 = -INFINITY;
                    tmem_ld64(tS, x, y);
                    if (masked) {
                        mask(x, vis[0]);
                        mask(y, vis[1]);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        top = fmaxf(top, x[e]);
                        top2 = fmaxf(top2, y[e]);
                    }
                    tmem_ld64(tS + 64, x, y);
                    if (masked) {
                        mask(x, vis[2]);
                        mask(y, vis[3]);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        top = fmaxf(top, x[e]);
                        top2 = fmaxf(top2, y[e]);
                    }
                    top = fmaxf(top, top2);
                    const bool grown = top != m && (top - m) * c > kSlack;
                    if (__any_sync(0xffffffffu, grown)) {
                        const float al = !grown ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - top) * c);
                        if (grown) m = top;
                        l *= al;
                        if (u > 0) {
                            if (!wait(&odone[i], (n - 1) & 1, budget)) {
                                ok = false;
                                break;
                            }
                            mma::tc_fence_after();
#pragma unroll 1
                            for (int j = 0; j < NB; ++j) {
                                float o[32];
                                mma::tmem_ld32_nowait(tO + 32 * j, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    uint32_t w[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[16 * h + e] * al);
                                    tmem_st16(tO + 32 * j + 16 * h, w);
                                }
                            }
                        }
                    }
                    // a row that has seen nothing has the maximum -infinity: its probabilities are zeros
                    const float mc = m == -INFINITY ? 0.0f : m * c;
                    float2 sum0 = make_float2(l, 0.0f), sum1 = make_float2(0.0f, 0.0f);
                    auto probs = [&](const float (&v)[32], uint32_t dst) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float2 d = __ffma2_rn(make_float2(v[e], v[e + 1]), make_float2(c, c), make_float2(-mc, -mc));
                            const float2 f = __ffma2_rn(make_float2(v[e + 2], v[e + 3]), make_float2(c, c), make_float2(-mc, -mc));
                            const float2 pd = make_float2(ex2(d.x), ex2(d.y)), pf = make_float2(ex2(f.x), ex2(f.y));
                            sum0 = __fadd2_rn(sum0, pd);
                            sum1 = __fadd2_rn(sum1, pf);
                            w[e / 2] = mma::pack_bf16x2(pd.x, pd.y);
                            w[e / 2 + 1] = mma::pack_bf16x2(pf.x, pf.y);
                        }
                        tmem_st16(dst, w);
                    };
                    probs(x, tP + 32);
                    probs(y, tP + 48);
                    tmem_ld64(tS, x, y);
                    if (masked) {
                        mask(x, vis[0]);
                        mask(y, vis[1]);
                    }
                    probs(x, tP);
                    probs(y, tP + 16);
                    l = (sum0.x + sum0.y) + (sum1.x + sum1.y);
                    tmem_wait_st();
                    mma::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pfull[i]);
                }
                if (!ok || !wait(&odone[i], (n - 1) & 1, budget)) {
                    ok = false;
                    break;
                }
                mma::tc_fence_after();
                const bool whole = count == units;
                float *sl = slot<R, D>(a, 2 * int(blockIdx.x) + (p.unit == 0 ? 1 : 0));
                const int ir = i * kTile + row;                              // row of the item
                const float inv = 1.0f / l;
                if (!whole && mine) {
                    sl[R * D + ir] = m == -INFINITY ? m : m * c;
                    sl[R * D + R + ir] = l;
                }
#pragma unroll 1
                for (int j = 0; j < NB; ++j) {
                    float o[32];
                    mma::tmem_ld32_nowait(tO + 32 * j, o);
                    tmem_wait_ld();
                    const bool nan = nan_first[seg % kSegs][j] < lim;
                    if (mine)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        // columns hold channels 0 4 1 5 2 6 3 7
                        float v[8] = {o[8 * g], o[8 * g + 2], o[8 * g + 4], o[8 * g + 6],
                                      o[8 * g + 1], o[8 * g + 3], o[8 * g + 5], o[8 * g + 7]};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (nan) v[e] = __uint_as_float(0x7fc00000u);
                            if (whole) v[e] = l == 0.0f && v[e] == 0.0f ? 0.0f : v[e] * inv;
                        }
                        if (whole) {
                            *reinterpret_cast<uint4 *>(a.out + (int64_t(q.lo + token) * a.hq + head) * D + 32 * j + 8 * g) =
                                make_uint4(mma::pack_bf16x2(v[0], v[1]), mma::pack_bf16x2(v[2], v[3]),
                                           mma::pack_bf16x2(v[4], v[5]), mma::pack_bf16x2(v[6], v[7]));
                        } else {
                            float *dst = sl + int64_t(ir) * D + 32 * j + 8 * g;
                            *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
                            *reinterpret_cast<float4 *>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
                }
                mma::tc_fence_before();
                if (tid == 0 && !whole && p.unit == 0) {
                    const int64_t last = total * (blockIdx.x + 1) / shares - left + units - 1;
                    int64_t e = blockIdx.x + 1;
                    while (total * (e + 1) / shares <= last) ++e;
                    *dsc = Desc{p.b, p.h, p.tile, int(e - blockIdx.x + 1)};
                }
            }
            k += count;
            left -= count;
            ++seg;
            if (left > 0) next_item<R>(a, q, p);
        }
    }

    mma::tc_fence_before();
    __syncthreads();
    if (warp == 15) {
        mma::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace chunk
}  // namespace attn
