// mx_chunk.cuh -- attention over the paged MXFP4 cache for many rows per kv
// head (chunks of prompts).  Included by kroquant.cu after mx_attention.cuh,
// whose division of the work it shares.
//
// An item is 256 consecutive rows of one (sequence, kv head): two tiles of 128
// rows.  For every step of 128 positions the fifth-generation tensor cores
// compute, for each tile,
//   S = Q K^T   (128 x 128, over the channels)       into tensor memory
//   O += P V    (128 x channels, over the positions) P from tensor memory
// with bf16 operands and fp32 sums, P = exp2(S c - m c).
//
// Bound: 4 D flops per row and position on the tensor cores and 16 exponentials
// per clock and SM: for D = 128 both take 1024 clocks per tile and step.  Tensor
// memory is full with S and O of two tiles (4 x 128 columns), so a tile's S
// cannot be computed ahead, and while one tile's softmax runs the tensor cores
// work for the other.  (S of 64 positions, twice for each tile, can be: but an
// MMA of 128 x 64 takes as long as one of 128 x 128, about 80 clocks, and the
// tensor cores became the limit.)
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
//             sum need no exchange.  P overwrites its S, the second 64 positions
//             first, and P V begins with them while the first 64 are computed.
//             O is rescaled only when a row's maximum has grown by more than 2^8
//             since the last time (exact: P and the sum use the same stale
//             maximum, and P <= 2^8 loses nothing in bf16).
//   8-14      decode: a step is 8 tasks, 32 positions of its keys or values each
//             (a lane per position), which the 7 warps take in turn
//   15        issues the MMAs: P0 V, Q0 K', P1 V, Q1 K' (K' the next step's)
// Q, K and V lie in the 128-byte swizzle, 64 channels to a row of 128 bytes; K
// and Q are read K-major, V with its channels as the major dimension.
// Every wait is bounded (g_wait_timeouts).
//
// Measured, 32 query heads over 8 of 128 channels: 2048 tokens over 32,048
// positions 0.93 ms in single replays, 1.12 PFLOP/s (0.68 of a cuBLAS bf16
// product's burst rate), 1.00 ms one after the other (0.75 of its sustained one);
// 512 over 8,512 88 us; a causal prompt of 4096 188 us.  A step of both tiles takes
// some 4200 clocks: tensor pipe and exponential
// unit 44 % busy, issue slots 50 %.  A tile's turn is Q K' (some 700 clocks with
// P V before it), the softmax (3000, of which 2000 while the other tile's
// exponentials compete), then P V.  An item costs some 12,000 clocks beside
// its steps: 3,500 until its queries are in place, 1,500 until the first S,
// 1,300 for the last P V, 4,400 for the results, 1,300 for the next item.

namespace attn {
namespace chunk {

constexpr int kTile = 128;                                   // rows of a tile
constexpr int kStep = 128;                                   // positions of a step
constexpr int R = 2 * kTile;                                 // rows of an item
constexpr int kSoftmaxWarps = 8;
constexpr int kRing = 2;                                     // steps of K and of V in shared memory
constexpr int kDecodeWarps = 7;
constexpr int kMmaWarp = kSoftmaxWarps + kDecodeWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
// Registers a thread: 128 at launch, some moved to the softmax warpgroups.  144 and 112, 152 and 104, 160 and 96: 512
// tokens after 30000 257, 260 and 258 us, 4096 fresh ones 194, 198 and 198.
constexpr int kSoftmaxRegs = 144, kOtherRegs = 112;
static_assert(kSoftmaxWarps % 4 == 0, "the split goes by whole warpgroups");
static_assert(kThreads == 512 && 256 * (kSoftmaxRegs + kOtherRegs) <= 512 * 128, "the split stays within the launch's registers");
constexpr int kSegs = 2 * kRing;                             // segments whose NaN positions are kept
constexpr int kItemCost = 4;                                 // of an item beside its units, in units
constexpr int kMergeQuads = 8;                               // channels / 4 that a CTA of the merge takes
constexpr int kMaxCtas = 192;                                // shares
constexpr float kSlack = 8.0f;                               // log2 of how far a maximum may be stale
// Values are summed at their full size, so sums over many large ones would pass fp32's range.  From this scale byte on
// (two bits in a byte) the probabilities of the rows that see one are taken 2^-48 smaller: below it 2^kSlack times 2^31
// values of 6 x 2^64 are still finite, from it on 2^31 of the largest; what gets lost is below 2^-78 of a row's largest
// probability or 2^-166 of the largest value.
constexpr uint32_t kLargeByte = 192;
constexpr float kLower = 48.0f;
constexpr uint32_t kO = 256;                                 // tensor memory: S of tile i at 128 i, O at 256 + 128 i
static_assert(kStep == kTile && kStep == kUnit, "S is square, a step is a unit");

template <int D_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr int NB = D / 32;
    static constexpr int kHalves = D > 64 ? 2 : 1;
    static constexpr int kQBytes = kHalves * kTile * 128;    // a tile of Q
    static constexpr int kStepBytes = kHalves * kStep * 128; // a step of K or V
    static constexpr int kSmem = 2 * kQBytes + 2 * kRing * kStepBytes + 1024;
    // kind::f16: fp32 sums, bf16 operands; S: N = 128, both K-major; O: N = D, B (bit 16) major in N
    static constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kStep >> 3) << 17) | (8u << 24);
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Where a warp is among the segments of its CTA's share.  It lives in shared
// memory: in registers it made the inner loops spill, and what is spilled comes
// back from L2, for shared memory leaves the first level little room.
struct Walk {
    Place p;
    Seq q;
    int64_t left;                            // units left, this segment's among them
    int count;                               // units of this segment
    int t_first, t_end, steps;               // its positions and steps
};

// Whole-warp wait on a barrier; false after the budget.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, long long budget)
{
    if (gemm::warp_wait(bar, parity, budget)) return true;
    if (threadIdx.x % 32 == 0) atomicAdd(&g_wait_timeouts, 1);
    return false;
}

// A value that all lanes hold, so that the compiler knows it: what the MMAs
// take then stays in uniform registers (moving each descriptor there for every
// MMA took more than the MMA).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }

// A position's codes and scale bytes of one array.
template <int NB>
struct Piece {
    uint4 c[NB];
    uint32_t s;                              // scale bytes
    uint32_t vs;                             // with keys: scale bytes of the values (load_vscales)
    bool on;                                 // within the segment and on a page
};

// Scale bytes of the values beside 32 keys (positions t .. t + 31, a position's pool row in each lane): two strips of
// 16 NB contiguous bytes, a word to each of the first 8 NB lanes.
template <int NB>
__device__ __forceinline__ uint32_t load_vscales(const uint8_t *__restrict__ scales, int64_t row)
{
    if constexpr (NB == 4) return row >= 0 ? __ldg(reinterpret_cast<const uint32_t *>(scales) + row) : 0u;
    const int lane = threadIdx.x % 32;
    const int64_t first = __shfl_sync(0xffffffffu, row, lane < 4 * NB ? 0 : 16);
    return lane < 8 * NB && first >= 0 ? __ldg(reinterpret_cast<const uint32_t *>(scales + first * NB) + lane % (4 * NB)) : 0u;
}

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

// A position into row `row` of the step at `dst`.  NaN blocks become NaN for
// keys and zeros for values, whose NaN is put into the result.
template <int NB>
__device__ __forceinline__ void decode_row(const Piece<NB> &p, uint32_t dst, int row, bool keys)
{
    const uint32_t sw = (row & 7) << 4;
    dst += row * 128;
    auto put = [&](int ch, uint4 v) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (ch / 8) * (kStep * 128) + (((ch % 8) << 4) ^ sw)),
                     "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
    };
    uint32_t top = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) top = max(top, (p.s >> (8 * b)) & 0xffu);
    // 2^(s - 1) as far as bf16 goes; a warp with a larger scale takes a second factor
    const bool large = __any_sync(0xffffffffu, top > 128u);
    if (!large) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t f = (((p.s >> (8 * b)) & 0xffu) + 126u) * 0x00800080u;
            put(4 * b, codes8_bf16(p.c[b].x, f));
            put(4 * b + 1, codes8_bf16(p.c[b].y, f));
            put(4 * b + 2, codes8_bf16(p.c[b].z, f));
            put(4 * b + 3, codes8_bf16(p.c[b].w, f));
        }
    } else {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t s = (p.s >> (8 * b)) & 0xffu;
            uint32_t f = (min(s, 128u) + 126u) * 0x00800080u, f2 = min(max(s, 128u) - 1u, 254u) * 0x00800080u;
            if (s >= kNanByte) {
                f = keys ? 0x3f803f80u : 0u;
                f2 = keys ? 0x7fc07fc0u : 0u;
            }
            auto twice = [&](uint32_t w) {
                const uint4 v = codes8_bf16(w, f);
                return make_uint4(hmul2_bf16(v.x, f2), hmul2_bf16(v.y, f2), hmul2_bf16(v.z, f2), hmul2_bf16(v.w, f2));
            };
            put(4 * b, twice(p.c[b].x));
            put(4 * b + 1, twice(p.c[b].y));
            put(4 * b + 2, twice(p.c[b].z));
            put(4 * b + 3, twice(p.c[b].w));
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
    __shared__ int64_t sh[kThreads + 34];
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) uint32_t visible[4][4];         // of step s % 4: the positions that are on a page, 32 to a word
    __shared__ int nan_first[kSegs][4];      // of segment i % kSegs, per 32 channels: the first position whose value is NaN
    __shared__ int large_first[kSegs];       // and the first with a large value
    __shared__ uint32_t lowered[kSoftmaxWarps];              // rows of a warp whose probabilities are taken smaller
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = base, *sK = base + 2 * C::kQBytes, *sV = sK + kRing * C::kStepBytes;
    __shared__ uint64_t kfull[kRing], kempty[kRing], vfull[kRing], vempty[kRing];
    __shared__ uint64_t qfull[2];            // Q of the tile in shared memory, the segment before put away
    __shared__ uint64_t sfull[2];            // S ready (and the P V before it done)
    __shared__ uint64_t pfull[4];            // [2 tile + half] P ready, O in order
    __shared__ uint64_t odone[2];            // the segment's last P V done
    __shared__ uint64_t segdone, done;       // a segment's MMAs done, all MMAs done
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
            mbar_init(&pfull[2 * i], 4);
            mbar_init(&pfull[2 * i + 1], 4);
            mbar_init(&odone[i], 1);
        }
        mbar_init(&segdone, 1);
        mbar_init(&done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __shared__ Walk walks[kThreads / 32];
    __shared__ int64_t totals[2];            // units of all shares, shares
    {
        Place p;
        int64_t total;
        int shares;
        const int64_t left = my_share<R, kItemCost, kThreads>(a, sh, p, total, shares);
        if (tid == 0) {
            reinterpret_cast<Desc *>(a.work)[blockIdx.x].parts = 0;
            totals[0] = total;
            totals[1] = shares;
        }
        if (left <= 0) return;
        if (lane == 0) {
            walks[warp].p = p;
            walks[warp].q = load_seq(a, p.b);
            walks[warp].left = left;
        }
    }
    if (tid < kSegs * 4) nan_first[tid / 4][tid % 4] = 0x7fffffff;
    if (tid < kSegs) large_first[tid] = 0x7fffffff;
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    mma::tc_fence_before();
    __syncthreads();
    mma::tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // Every role walks the same segments: units [p.unit, p.unit + count) of item (b, h, tile), that is the
    // positions from t_first up to t_end in `steps` steps.
    Walk &walk = walks[warp];
    int seg = 0;                             // segments so far
    auto segment = [&] {
        if (lane == 0) {
            const Place p = walk.p;
            const Seq q = walk.q;
            const int count = int(min(walk.left, int64_t(item_units<R>(a, q, p.tile) - p.unit)));
            walk.count = count;
            walk.t_first = p.unit * kUnit;
            walk.t_end = min(row_end(a, q, min((p.tile + 1) * R, q.rows) - 1), walk.t_first + count * kUnit);
            walk.steps = max((walk.t_end - walk.t_first + kStep - 1) / kStep, 1);
        }
        __syncwarp();
    };
    auto advance = [&] {
        __syncwarp();
        if (lane == 0) {
            walk.left -= walk.count + kItemCost;
            if (walk.left > 0) {
                Place p = walk.p;
                Seq q = walk.q;
                next_item<R>(a, q, p);
                walk.p = p;
                walk.q = q;
            }
        }
        __syncwarp();
        ++seg;
    };
    // All warps of a warpgroup execute the same setmaxnreg: warps 12 to 15 have two roles, so theirs stands before
    // the roles.  (The softmax warps' there, too, makes their loops spill.)
    if (warp >= kSoftmaxWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp >= kSoftmaxWarps && warp < kMmaWarp) {
        // ---------------- keys and values into shared memory
        int k = 0;                           // steps of the segments so far
        int turn = warp - kSoftmaxWarps;                 // this warp's next task, counted from the segment's first
        bool ok = true;
        while (walk.left > 0 && ok) {
            segment();
            const int32_t *table = a.s.table + int64_t(walk.p.b) * a.s.table_stride;
            const int t_first = walk.t_first, t_end = walk.t_end, steps = walk.steps, head = walk.p.h;
            const int tasks = steps * 8;
            // task x: step x / 8, values if x & 4, positions 32 (x & 3) + lane.  The pages are looked up one task
            // ahead of the codes, the codes one task ahead of their use.
            auto page_index = [&](int t) { return a.page_shift >= 0 ? t >> a.page_shift : t / a.s.page; };
            auto position = [&](int x) { return t_first + (x >> 3) * kStep + 32 * (x & 3) + lane; };
            auto page_of = [&](int x) -> int {
                const int64_t t = int64_t(t_first) + int64_t(x >> 3) * kStep + 32 * (x & 3) + lane;
                return t < t_end ? __ldg(table + page_index(int(t))) : -1;
            };
            auto load = [&](Piece<NB> &v, int x, int page) {
                const int t = position(x);
                const bool is_v = x & 4;
                int64_t row = -1;
                if (page >= 0 && page < a.s.num_pages)
                    row = (int64_t(page) * a.s.heads + head) * a.s.page + (t - page_index(t) * a.s.page);
                load_piece<NB>(v, is_v ? a.vc : a.kc, is_v ? a.vs : a.ks, row);
                if (!is_v) v.vs = load_vscales<NB>(a.vs, row);
            };
            Piece<NB> next;
            load(next, turn, page_of(turn));
            int ahead = page_of(turn + kDecodeWarps);
            int x = turn;
            for (; x < tasks; x += kDecodeWarps) {
                const Piece<NB> cur = next;
                load(next, x + kDecodeWarps, ahead);
                ahead = page_of(x + 2 * kDecodeWarps);
                const int u = x >> 3, part = x & 3, ku = k + u, st = ku % kRing, row = 32 * part + lane;
                const bool is_v = x & 4;
                if (ku >= kRing && !wait(is_v ? &vempty[st] : &kempty[st], ((ku / kRing) - 1) & 1, budget)) {
                    ok = false;
                    break;
                }
                if (is_v) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        if (((cur.s >> (8 * b)) & 0xffu) >= kNanByte)
                            atomicMin(&nan_first[seg % kSegs][b], t_first + u * kStep + row);
                } else {
                    const uint32_t on = __ballot_sync(0xffffffffu, cur.on);
                    if (lane == 0) visible[ku & 3][part] = on;
                    // the values' scales with the keys, for the softmax has to know before it makes probabilities
                    if (cur.vs & (cur.vs << 1) & 0x80808080u) {
#pragma unroll 1
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t sb = (cur.vs >> (8 * e)) & 0xffu;
                            const int t = t_first + u * kStep + 32 * part + 16 * (lane / (4 * NB)) + (4 * (lane % (4 * NB)) + e) / NB;
                            if (sb >= kLargeByte && sb < kNanByte && t < t_end) atomicMin(&large_first[seg % kSegs], t);
                        }
                    }
                }
                decode_row<NB>(cur, smem_addr(is_v ? sV : sK) + st * C::kStepBytes, row, !is_v);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(is_v ? &vfull[st] : &kfull[st]);
            }
            turn = x - tasks;
            k += steps;
            advance();
        }
    } else if (warp == kMmaWarp) {
        // ---------------- the MMAs
        int k = 0, n1 = 0;                   // steps, steps of the second tile so far
        bool ok = true;
        const uint32_t tm = uniform(tmem), aQ = uniform(smem_addr(sQ));
        const uint32_t aK = aQ + 2 * C::kQBytes, aV = aK + kRing * C::kStepBytes;
        auto qk = [&](int i, int st) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                umma_ss(tm + i * 128, desc(aQ + i * C::kQBytes + (j / 4) * (kTile * 128) + (j % 4) * 32, 16),
                        desc(aK + st * C::kStepBytes + (j / 4) * (kStep * 128) + (j % 4) * 32, 16), C::kIdescS, j > 0);
            gemm::umma_commit_w(&sfull[i]);
        };
        auto pv = [&](int i, int st, int half, bool add) {
#pragma unroll
            for (int j = 4 * half; j < 4 * half + 4; ++j)    // P: 32 columns in either half of S
                umma_ts(tm + kO + i * 128, tm + i * 128 + half * 64 + (j % 4) * 8,
                        desc(aV + st * C::kStepBytes + j * 16 * 128, kStep * 128), C::kIdescO, add || j > 4 * half);
        };
        while (uniform(walk.left > 0) && ok) {
            segment();
            const int n = int(uniform(uint32_t(walk.steps)));
            const bool two = uniform(walk.q.rows - walk.p.tile * R > kTile);
            if (!wait(&kfull[k % kRing], (k / kRing) & 1, budget) || !wait(&qfull[0], seg & 1, budget) ||
                !wait(&qfull[1], seg & 1, budget))
                break;
            mma::tc_fence_after();
            qk(0, k % kRing);
            if (two) qk(1, k % kRing);
            gemm::umma_commit_w(&kempty[k % kRing]);
            for (int u = 0; u < n && ok; ++u, ++k) {
                const int st = k % kRing, sn = (k + 1) % kRing;
                const bool more = u + 1 < n;
                ok = wait(&vfull[st], (k / kRing) & 1, budget) && wait(&pfull[1], k & 1, budget);
                if (!ok) break;
                mma::tc_fence_after();
                pv(0, st, 1, u > 0);
                ok = wait(&pfull[0], k & 1, budget);
                if (!ok) break;
                mma::tc_fence_after();
                pv(0, st, 0, true);
                if (!two) gemm::umma_commit_w(&vempty[st]);
                if (more) {
                    ok = wait(&kfull[sn], ((k + 1) / kRing) & 1, budget);
                    if (!ok) break;
                    mma::tc_fence_after();
                    qk(0, sn);
                } else {
                    gemm::umma_commit_w(&odone[0]);
                }
                if (two) {
                    ok = wait(&pfull[3], n1 & 1, budget);
                    if (!ok) break;
                    mma::tc_fence_after();
                    pv(1, st, 1, u > 0);
                    ok = wait(&pfull[2], n1 & 1, budget);
                    if (!ok) break;
                    ++n1;
                    mma::tc_fence_after();
                    pv(1, st, 0, true);
                    gemm::umma_commit_w(&vempty[st]);
                    if (more) qk(1, sn);
                    else gemm::umma_commit_w(&odone[1]);
                }
                if (more) gemm::umma_commit_w(&kempty[sn]);
            }
            if (!ok) break;
            gemm::umma_commit_w(&segdone);
            advance();
        }
        // every MMA issued has completed before the tensor memory is freed
        gemm::umma_commit_w(&done);
        wait(&done, 0, budget);
    } else {
        // ---------------- softmax: thread = row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int i = warp / 4, row = tid % kTile;
        const uint32_t lanes = uint32_t(warp % 4) << 21;                     // 32 (warp % 4) in the lane field
        uint8_t *tile_q = sQ + i * C::kQBytes;
        const uint32_t tS = tmem + lanes + i * 128, tO = tmem + lanes + kO + i * 128;
        int n = 0;                           // steps of this tile so far
        int k = 0;                           // steps so far
        int mine_segs = 0;                   // segments of this tile so far
        const float c = a.scale_log2 == 0.0f ? 1.0f : fabsf(a.scale_log2);
        bool ok = true;
        // The lane for places in Q and in the results.  With 12 chunks to a row the places cost divisions and would
        // be kept from item to item, which spills: from a lane that looks new they are worked out again (2 x 777 of
        // 3000, 96 channels: 92.6 -> 83.4 us; with 16 chunks 55.8 -> 59.3 us, so there they are not).
        auto fresh_lane = [&] {
            int ln = lane;
            if constexpr (NB == 3) asm volatile("" : "+r"(ln));
            return ln;
        };
        while (walk.left > 0 && ok) {
            segment();
            const int steps = walk.steps;
            const int r0 = walk.p.tile * R + i * kTile;
            // Keys and values run kRing steps, so at most kRing segments ahead: nobody writes this slot before this
            // segment's P V, and who read it (kRing segments ago) is through, since a segment's first MMA waits
            // for both tiles' softmax.
            if (tid < 4) nan_first[(seg + kRing) % kSegs][tid] = 0x7fffffff;
            if (tid == 0) large_first[(seg + kRing) % kSegs] = 0x7fffffff;
            if (lane == 0) lowered[warp] = 0;
            if (r0 >= walk.q.rows) {
                // nothing to do, but the next segment begins after both tiles' last
                __syncwarp();
                if (lane == 0) mbar_arrive(&qfull[i]);
            } else {
                // positions from the step's first that the row sees; one that is not there sees all, for nothing
                int lim;
                // Q: rows of the tile, channels of 8 in the decoders' order; the sign (or zero) of the scale
                // goes into it
                {
                    const Seq q = walk.q;
                    const int r = r0 + row, rc = min(r, q.rows - 1), token = rc / a.group;
                    lim = r < q.rows ? row_end(a, q, r) - walk.t_first : 0x7fffffff;
                    const int64_t from = int64_t(q.lo + token) * a.q_st +
                                         int64_t(walk.p.h * a.group + rc - token * a.group) * a.q_sh;
                    const uint32_t sgn = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
                    const bool zero = a.scale_log2 == 0.0f;
                    // lanes over the chunks of the warp's rows, so that every load is contiguous, and all loads
                    // before the first use: one after the other they took 13k cycles an item, together 3.5k.  A row
                    // that is not there reads the last one's, for nothing.
                    const int ln = fresh_lane();
                    uint4 w[D / 8];
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) {
                        const int pc = ln + 32 * e, rr = pc / (D / 8), ch = pc % (D / 8);
                        w[e] = __ldg(reinterpret_cast<const uint4 *>(a.q + __shfl_sync(0xffffffffu, from, rr)) + ch);
                    }
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) {
                        const int pc = ln + 32 * e, rr = pc / (D / 8), ch = pc % (D / 8), rw = row - ln + rr;
                        if (zero)
                            w[e] = make_uint4(hmul2_bf16(w[e].x, 0u), hmul2_bf16(w[e].y, 0u), hmul2_bf16(w[e].z, 0u),
                                              hmul2_bf16(w[e].w, 0u));
                        *reinterpret_cast<uint4 *>(tile_q + rw * 128 + (ch / 8) * (kTile * 128) + (((ch % 8) ^ (rw & 7)) << 4)) =
                            make_uint4(__byte_perm(w[e].x, w[e].z, 0x5410) ^ sgn, __byte_perm(w[e].x, w[e].z, 0x7632) ^ sgn,
                                       __byte_perm(w[e].y, w[e].w, 0x5410) ^ sgn, __byte_perm(w[e].y, w[e].w, 0x7632) ^ sgn);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&qfull[i]);
                }
                int lim_min = __reduce_min_sync(0xffffffffu, lim);     // of the warp's rows
                float m = -INFINITY, l = 0.0f;                               // the maximum in use, the sum
                for (int u = 0; u < steps; ++u, ++n, lim -= kStep, lim_min -= kStep) {
                    if (!wait(&sfull[i], n & 1, budget)) {
                        ok = false;
                        break;
                    }
                    mma::tc_fence_after();
                    const uint32_t *on = visible[(k + u) & 3];
                    float x[32], y[32];
                    const uint4 all = *reinterpret_cast<const uint4 *>(on);
                    if (lim_min < kStep || (all.x & all.y & all.z & all.w) != 0xffffffffu) {
                        // rare: what the rows do not see becomes -infinity in tensor memory
#pragma unroll 1
                        for (int j = 0; j < 4; ++j) {
                            const int see = lim - 32 * j;
                            const uint32_t bits = on[j] & (see >= 32 ? 0xffffffffu : see <= 0 ? 0u : (1u << see) - 1u);
                            mma::tmem_ld32_nowait(tS + 32 * j, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t w[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    w[e] = (bits >> (16 * h + e)) & 1 ? __float_as_uint(x[16 * h + e]) : 0xff800000u;
                                tmem_st16(tS + 32 * j + 16 * h, w);
                            }
                        }
                        tmem_wait_st();
                    }
                    float top = m, top2 = -INFINITY;
                    auto maximum = [&](uint32_t src) {
                        mma::tmem_ld32_nowait(src, x);
                        mma::tmem_ld32_nowait(src + 32, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            top = fmaxf(fmaxf(top, x[e]), x[e + 1]);
                            top2 = fmaxf(fmaxf(top2, y[e]), y[e + 1]);
                        }
                    };
                    maximum(tS);
                    maximum(tS + 64);
                    top = fmaxf(top, top2);
                    const bool grown = top != m && (top - m) * c > kSlack;
                    // (this step's keys have been decoded, so its large values are known)
                    const int large = *const_cast<volatile int *>(&large_first[seg % kSegs]);
                    float lower = 0.0f;
                    if (__any_sync(0xffffffffu, grown || large != 0x7fffffff)) {
                        float al = !grown ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - top) * c);
                        if (grown) m = top;
                        if (large != 0x7fffffff) {           // rarest: rows that see it, from now on or before
                            const bool sees = large - (walk.t_first + u * kStep) < lim;
                            if (sees) lower = kLower;
                            if (sees && !((lowered[warp] >> lane) & 1)) al *= ex2(-kLower);
                            const uint32_t now = __ballot_sync(0xffffffffu, sees);
                            if (lane == 0) lowered[warp] = now;
                            __syncwarp();
                        }
                        l *= al;
                        if (u > 0) {
#pragma unroll 1
                            for (int j = 0; j < 2 * NB; ++j) {
                                float o[16];
                                tmem_ld16(tO + 16 * j, o);
                                tmem_wait_ld();
                                uint32_t w[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * al);
                                tmem_st16(tO + 16 * j, w);
                            }
                        }
                    }
                    // a row that has seen nothing has the maximum -infinity: its probabilities are zeros
                    const float mc = m == -INFINITY ? 0.0f : fmaf(m, c, lower);
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
                    auto ready = [&](int half) {
                        tmem_wait_st();
                        mma::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&pfull[2 * i + half]);
                    };
                    probs(x, tS + 64);
                    probs(y, tS + 80);
                    ready(1);
                    mma::tmem_ld32_nowait(tS, x);
                    mma::tmem_ld32_nowait(tS + 32, y);
                    tmem_wait_ld();
                    probs(x, tS);
                    probs(y, tS + 16);
                    l = (sum0.x + sum0.y) + (sum1.x + sum1.y);
                    ready(0);
                }
                if (!ok || !wait(&odone[i], mine_segs++ & 1, budget)) {
                    ok = false;
                    break;
                }
                mma::tc_fence_after();
                const Seq q = walk.q;
                const Place p = walk.p;
                const int r = p.tile * R + i * kTile + row;
                const bool mine = r < q.rows;
                const int sees = mine ? row_end(a, q, r) : 0;
                const int units = item_units<R>(a, q, p.tile);
                const bool whole = walk.count == units;
                float *sl = slot<R, D>(a, 2 * int(blockIdx.x) + (p.unit == 0 ? 1 : 0));
                const int ir = i * kTile + row;                              // row of the item
                float scale = 1.0f / l;
                if (l == 0.0f) scale = whole && mine ? empty_row(a, p.b, sees) : 0.0f;
                if (!whole && mine) {
                    const float lower = (lowered[warp] >> lane) & 1 ? kLower : 0.0f;
                    sl[R * D + ir] = m == -INFINITY ? m : fmaf(m, c, lower);
                    sl[R * D + R + ir] = l;
                }
#pragma unroll 1
                for (int j = 0; j < NB; ++j) {
                    float o[32];
                    mma::tmem_ld32_nowait(tO + 32 * j, o);
                    const float f = nan_first[seg % kSegs][j] < sees ? __uint_as_float(0x7fc00000u) : scale;
                    tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        // columns hold channels 0 4 1 5 2 6 3 7; the sum makes a negative zero positive
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = fmaf(o[8 * h + 2 * (e % 4) + e / 4], f, 0.0f);
                        const int ch = 4 * j + h;                            // of 8 channels
                        if (whole) {
                            // by way of Q's place, which the segment has done with, so that rows are written whole
                            *reinterpret_cast<uint4 *>(tile_q + row * 128 + (ch / 8) * (kTile * 128) + (((ch % 8) ^ (row & 7)) << 4)) =
                                make_uint4(mma::pack_bf16x2(v[0], v[1]), mma::pack_bf16x2(v[2], v[3]),
                                           mma::pack_bf16x2(v[4], v[5]), mma::pack_bf16x2(v[6], v[7]));
                        } else if (mine) {
                            *reinterpret_cast<float4 *>(sl + slot_at<R>(ir, 8 * ch)) = make_float4(v[0], v[1], v[2], v[3]);
                            *reinterpret_cast<float4 *>(sl + slot_at<R>(ir, 8 * ch + 4)) = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
                }
                __syncwarp();
                if (whole) {
                    const int token = r / a.group;
                    const int ln = fresh_lane();
                    const int64_t to = (int64_t(q.lo + token) * a.hq + p.h * a.group + r - token * a.group) * D;
#pragma unroll 1
                    for (int e0 = 0; e0 < D / 8; e0 += 4) {
                        uint4 w[4];
                        int64_t at[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int pc = ln + 32 * (e0 + e), rr = pc / (D / 8), ch = pc % (D / 8), rw = row - ln + rr;
                            w[e] = *reinterpret_cast<const uint4 *>(tile_q + rw * 128 + (ch / 8) * (kTile * 128) + (((ch % 8) ^ (rw & 7)) << 4));
                            at[e] = __shfl_sync(0xffffffffu, to, rr) + 8 * ch;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int rr = (ln + 32 * (e0 + e)) / (D / 8);
                            if (r0 + row - ln + rr < q.rows) *reinterpret_cast<uint4 *>(a.out + at[e]) = w[e];
                        }
                    }
                    __syncwarp();
                }
                mma::tc_fence_before();
                if (tid == 0 && !whole && p.unit == 0) {
                    const int64_t total = totals[0], shares = totals[1];
                    const int64_t end = quotient(total * (blockIdx.x + 1), shares) - walk.left + units - 1;
                    reinterpret_cast<Desc *>(a.work)[blockIdx.x] =
                        Desc{int(share_of(end, total, shares)) - int(blockIdx.x) + 1, p.h, p.tile * R, q.lo, q.rows, p.b, {}};
                }
            }
            // A tile's arrivals must not run ahead of the segments.  Both tiles wait in every segment: a wait on
            // phase n passes also while phase n - 1 is not complete, so none may be left out.
            if (!wait(&segdone, seg & 1, budget)) break;
            k += steps;
            advance();
        }
    }

    mma::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        mma::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// The items that were split, as in merge_kernel, for many rows and (mostly) two
// parts: a thread per row and 16 channels, which finds its row's weights itself
// and has the first two parts' values on their way meanwhile.
template <int D>
__global__ void __launch_bounds__(2 * R)
merge_many_kernel(const Args a)
{
    pdl_wait();
    constexpr int kPer = kMergeQuads / 2;                    // quads of a thread
    const int share = int(blockIdx.x) / (D / 4 / kMergeQuads), r = threadIdx.x % R;
    const int quad = int(blockIdx.x) % (D / 4 / kMergeQuads) * kMergeQuads + int(threadIdx.x) / R * kPer;
    const Desc d = reinterpret_cast<const Desc *>(a.work)[share];
    if (d.parts == 0 || d.r0 + r >= d.rows) return;
    auto part = [&](int k) { return slot<R, D>(a, k ? 2 * (share + k) : 2 * share + 1); };
    auto load = [&](float4 (&v)[kPer], int k) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = *reinterpret_cast<const float4 *>(part(k) + slot_at<R>(r, 4 * (quad + j)));
    };
    float4 v0[kPer], v1[kPer];
    load(v0, 0);                                             // (two parts at least)
    load(v1, 1);
    float mm = -INFINITY, ll = 0.0f;
    for (int k = 0; k < d.parts; ++k) mm = fmaxf(mm, part(k)[R * D + r]);
    auto weight = [&](int k) {
        const float mk = part(k)[R * D + r], lk = part(k)[R * D + R + r];
        // a part that saw nothing has nothing; a NaN sum reaches the result
        return mk == -INFINITY ? (lk == 0.0f ? 0.0f : lk) : lk * ex2(mk - mm);
    };
    for (int k = 0; k < d.parts; ++k) ll += weight(k);
    const float inv = ll == 0.0f ? empty_row(a, d.b, row_end(a, load_seq(a, d.b), d.r0 + r)) : 1.0f / ll;
    float4 x[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = 0; k < d.parts; ++k) {
        const float f = weight(k) * inv;                     // its share of the sum
        float4 v[kPer];
        if (k > 1) load(v, k);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float4 u = k == 0 ? v0[j] : k == 1 ? v1[j] : v[j];
            x[j].x = fmaf(u.x, f, x[j].x);
            x[j].y = fmaf(u.y, f, x[j].y);
            x[j].z = fmaf(u.z, f, x[j].z);
            x[j].w = fmaf(u.w, f, x[j].w);
        }
    }
    const int row = d.r0 + r, token = row / a.group;
    __nv_bfloat16 *out = a.out + (int64_t(d.lo + token) * a.hq + d.h * a.group + row - token * a.group) * D + 4 * quad;
#pragma unroll
    for (int j = 0; j < kPer; j += 2) {
        *reinterpret_cast<uint4 *>(out + 4 * j) =
            make_uint4(mma::pack_bf16x2(x[j].x, x[j].y), mma::pack_bf16x2(x[j].z, x[j].w),
                       mma::pack_bf16x2(x[j + 1].x, x[j + 1].y), mma::pack_bf16x2(x[j + 1].z, x[j + 1].w));
    }
}

}  // namespace chunk
}  // namespace attn
