// mx_cache.cuh -- a paged MXFP4 cache of keys and values: quantized as it is
// written, and read back.  Included by kroquant.cu; uses its helpers.
//
// A cache is a pool of pages; page p holds page_size positions of every kv
// head, codes [num_pages][heads][page_size][D/2] and scales
// [num_pages][heads][page_size][D/32].  A page's positions of one head are
// contiguous, so attention over the cache streams them, and 16 of them begin
// on a 16-byte boundary in both arrays.
//
// Rows of a call (new tokens, or positions to read) are packed sequence after
// sequence: rows cu[b] .. cu[b+1] belong to sequence b.  Everything that the
// device arrays say is bounded here before it is used, so a plan that is
// wrong costs rows, never an access out of bounds.

__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight codes as bf16 pairs (0,4) (1,5) (2,6) (3,7), times the pair f: one AND,
// one multiply and one AND put codes n and n + 4 side by side as bf16 numbers
// code * 2^-126 (code 1, 0.5, is a subnormal).
__device__ __forceinline__ uint4 codes8_bf16(uint32_t w, uint32_t f)
{
    constexpr uint32_t kA = (1u << 12) + (1u << 6), kB = (1u << 8) + (1u << 2), kM = 0x81C081C0u;
    const uint32_t v = w >> 8;
    return make_uint4(hmul2_bf16(((w & 0x000F000Fu) * kA) & kM, f), hmul2_bf16(((w & 0x00F000F0u) * kB) & kM, f),
                      hmul2_bf16(((v & 0x000F000Fu) * kA) & kM, f), hmul2_bf16(((v & 0x00F000F0u) * kB) & kM, f));
}

namespace cache {

// The device arrays of a call's sequences (mx_batch of the header).
struct Seqs {
    const int32_t *table;      // [B][table_stride], page of every page_size positions
    int64_t table_stride;
    const int32_t *cu;         // [B + 1]
    const int32_t *len;        // [B] (may be NULL where a call does not read it)
    int B;
    int T;                     // rows of the call
    int max_pages;             // entries of a table row
    int num_pages;
    int page;                  // positions per page
    int heads;                 // kv heads
};

// Rows of sequence b: [lo, hi) within [0, T).
__device__ __forceinline__ void seq_rows(const Seqs &s, int b, int &lo, int &hi)
{
    lo = max(0, min(__ldg(s.cu + b), s.T));
    hi = max(lo, min(__ldg(s.cu + b + 1), s.T));
}

// Positions of sequence b that its table row can hold.
__device__ __forceinline__ int64_t seq_cap(const Seqs &s) { return int64_t(s.max_pages) * s.page; }

// The sequence of row t: the last b with cu[b] <= t < cu[b+1]; -1 where no
// sequence has the row (padding behind the last).
__device__ __forceinline__ int seq_of_row(const Seqs &s, int t)
{
    int lo = 0, hi = s.B;                    // the first b in [0, B] with cu[b] > t, less one
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(s.cu + mid) <= t) lo = mid + 1;
        else hi = mid;
    }
    const int b = lo - 1;
    return b >= 0 && t < __ldg(s.cu + b + 1) ? b : -1;
}

// Index of position pos of sequence b, head h among the pool's
// (page, head, position) rows; -1 where the table names no page of the pool.
__device__ __forceinline__ int64_t cache_row(const Seqs &s, int b, int h, int64_t pos)
{
    if (pos < 0 || pos >= seq_cap(s)) return -1;
    const int j = int(pos / s.page);
    const int p = __ldg(s.table + int64_t(b) * s.table_stride + j);
    if (p < 0 || p >= s.num_pages) return -1;
    return (int64_t(p) * s.heads + h) * s.page + (pos - int64_t(j) * s.page);
}

// Both kernels: a warp per token and array, a lane per 8 channels (a block of 32
// is 4 neighbouring lanes), so that every access of a warp is contiguous but for
// the heads' distance in the pool, and what finds the token's place is done once
// for heads x D channels.  Up to kPieces loads of a lane are in flight.  Bound by
// the bytes read and written: 75,149 positions of 8 heads x 128 channels back as
// bf16 in 71 us, 5.5 TB/s; 18,731 fp32 tokens into the cache and back in 56 us, 32
// of them the write, 5.4 TB/s.  (A thread per 32-block took 104 and 74 us.)
constexpr int kPieces = 4;

// Place of row t: its sequence's pool row for head 0 (-1 if on no page), or no
// sequence (false).  Position: the last new tokens' (len) or from `starts`.
__device__ __forceinline__ bool row_place(const Seqs &s, int t, const int32_t *starts, bool read, int64_t &row)
{
    const int b = seq_of_row(s, t);
    if (b < 0) return false;
    int lo, hi;
    seq_rows(s, b, lo, hi);
    const int64_t pos = read ? int64_t(t - lo) + (starts ? __ldg(starts + b) : 0) : int64_t(__ldg(s.len + b)) - hi + t;
    row = cache_row(s, b, 0, pos);
    return true;
}

// A lane's pieces p0, p0 + 32, ...: 32 pieces are whole heads (but for three
// blocks to a head), so that a place is the first one's and a multiple of a
// stride: what finds it was most of the instructions otherwise.
template <int NB>
struct Lane {
    static constexpr int PH = 4 * NB;        // pieces of a head
    int h, c;                                // head and place in it of piece p0

    __device__ __forceinline__ Lane(int p0) : h(p0 / PH), c(p0 % PH) {}
    // for piece p0 + 32 i: the number of heads further, and the place
    __device__ __forceinline__ int heads(int i) const { return 32 % PH == 0 ? i * (32 / PH) : (c + 32 * i) / PH; }
    __device__ __forceinline__ int place(int i) const { return 32 % PH == 0 ? c : (c + 32 * i) % PH; }
};

// Eight codes as bf16 pairs in order, times 2^(sb - 127); NaN for 255.  (Exact; as
// two factors, for bf16 takes code * 2^-126 to at most code * 2 in one.)
__device__ __forceinline__ uint4 decode_bf16(uint32_t w, uint32_t sb)
{
    uint4 x = codes8_bf16(w, (min(sb, 128u) + 126u) * 0x00800080u);
    if (sb > 128u) {
        const uint32_t f2 = sb == 255u ? 0x7fc07fc0u : (sb - 1u) * 0x00800080u;
        x = make_uint4(hmul2_bf16(x.x, f2), hmul2_bf16(x.y, f2), hmul2_bf16(x.z, f2), hmul2_bf16(x.w, f2));
    }
    return make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.z, x.w, 0x5410), __byte_perm(x.x, x.y, 0x7632),
                      __byte_perm(x.z, x.w, 0x7632));
}

// Quantize the keys and values of new tokens into the cache, as the other MXFP4
// kernels do: the four lanes of a block share its largest magnitude (bits order
// like magnitudes, and what is not finite is above all that is).
template <bool F32, int NB>
__global__ void __launch_bounds__(kThreads)
write_kernel(const void *__restrict__ k, const void *__restrict__ v, int64_t kst, int64_t ksh, int64_t vst,
             int64_t vsh, uint32_t *__restrict__ kc, uint8_t *__restrict__ ks, uint32_t *__restrict__ vc,
             uint8_t *__restrict__ vs, Seqs s)
{
    pdl_wait();
    constexpr int PH = 4 * NB;                               // pieces of a head
    const int lane = threadIdx.x % 32, pieces = s.heads * PH;
    const int64_t warps = int64_t(gridDim.x) * (kThreads / 32);
    for (int64_t task = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; task < 2 * int64_t(s.T); task += warps) {
        const int t = int(task >> 1);
        const bool is_v = task & 1;
        int64_t row;
        if (!row_place(s, t, nullptr, false, row) || row < 0) continue;
        const int64_t sh = is_v ? vsh : ksh, src = int64_t(t) * (is_v ? vst : kst);
        const void *in = is_v ? v : k;
        uint32_t *codes = is_v ? vc : kc;
        uint8_t *scales = is_v ? vs : ks;
        for (int p0 = lane; p0 - lane < pieces; p0 += 32 * kPieces) {
            const Lane<NB> of(p0);
            const int64_t src0 = src + of.h * sh, row0 = row + int64_t(of.h) * s.page;
            float x[kPieces][8];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int64_t at = src0 + of.heads(i) * sh + 8 * of.place(i);
                if (p0 + 32 * i < pieces) {
                    if constexpr (F32) {
                        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(in) + at);
                        const float4 u = __ldg(q), w = __ldg(q + 1);
                        x[i][0] = u.x, x[i][1] = u.y, x[i][2] = u.z, x[i][3] = u.w;
                        x[i][4] = w.x, x[i][5] = w.y, x[i][6] = w.z, x[i][7] = w.w;
                    } else {
                        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(in) + at));
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[i][2 * e] = bf16_lo(w[e]), x[i][2 * e + 1] = bf16_hi(w[e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int c = of.place(i);
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[i][e]) & 0x7fffffffu);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (p0 + 32 * i >= pieces) continue;
                uint32_t sb = 0xFFu, w = 0;
                if (top < 0x7f800000u) {
                    sb = e8m0_byte(__uint_as_float(top));
                    const float f = inv_scale(sb);
                    w = cvt_e2m1x8(x[i][0] * f, x[i][1] * f, x[i][2] * f, x[i][3] * f, x[i][4] * f, x[i][5] * f, x[i][6] * f,
                                   x[i][7] * f);
                }
                const int64_t to = row0 + of.heads(i) * int64_t(s.page);
                codes[to * PH + c] = w;
                if (c % 4 == 0) scales[to * NB + c / 4] = uint8_t(sb);
            }
        }
    }
}

// Positions starts[b] + (row - cu[b]) of every sequence, decoded to bf16
// (exact but for overflow: two significant bits times a power of two) or
// fp32.  Rows that the table names no page for come out as zeros.
template <bool F32, int NB>
__global__ void __launch_bounds__(kThreads)
read_kernel(const uint32_t *__restrict__ kc, const uint8_t *__restrict__ ks, const uint32_t *__restrict__ vc,
            const uint8_t *__restrict__ vs, const int32_t *__restrict__ starts, void *__restrict__ out_k,
            void *__restrict__ out_v, Seqs s)
{
    pdl_wait();
    constexpr int PH = 4 * NB;
    const int lane = threadIdx.x % 32, pieces = s.heads * PH;
    const int64_t warps = int64_t(gridDim.x) * (kThreads / 32);
    for (int64_t task = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; task < 2 * int64_t(s.T); task += warps) {
        const int t = int(task >> 1);
        const bool is_v = task & 1;
        int64_t row;
        if (!row_place(s, t, starts, true, row)) continue;
        const uint32_t *codes = is_v ? vc : kc;
        const uint8_t *scales = is_v ? vs : ks;
        void *out = is_v ? out_v : out_k;
        for (int p0 = lane; p0 < pieces; p0 += 32 * kPieces) {
            const Lane<NB> of(p0);
            const int64_t row0 = row + int64_t(of.h) * s.page;
            uint32_t w[kPieces], sb[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                w[i] = sb[i] = 0;
                if (p0 + 32 * i < pieces && row >= 0) {
                    const int64_t at = row0 + of.heads(i) * int64_t(s.page);
                    w[i] = __ldg(codes + at * PH + of.place(i));
                    sb[i] = __ldg(scales + at * NB + of.place(i) / 4);
                }
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int p = p0 + 32 * i;
                if (p >= pieces) break;
                const int64_t to = int64_t(t) * pieces + p;
                if constexpr (F32) {
                    const float f = e8m0_value(sb[i]);
                    float2 e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e[j] = e2m1x2_to_f32x2((w[i] >> (8 * j)) & 0xFFu);
                        e[j].x *= f;
                        e[j].y *= f;
                    }
                    float4 *o = static_cast<float4 *>(out) + to * 2;
                    o[0] = make_float4(e[0].x, e[0].y, e[1].x, e[1].y);
                    o[1] = make_float4(e[2].x, e[2].y, e[3].x, e[3].y);
                } else {
                    static_cast<uint4 *>(out)[to] = decode_bf16(w[i], sb[i]);
                }
            }
        }
    }
}

}  // namespace cache
