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

// Quantize the keys and values of new tokens into the cache.  One thread per
// 32-block: it reads 64 (128) bytes of its row, quantizes them as the other
// MXFP4 kernels do and writes 16 bytes of codes and the scale byte.  Bound by
// the bytes read and written.
template <bool F32>
__global__ void __launch_bounds__(kThreads)
write_kernel(const void *__restrict__ k, const void *__restrict__ v, int64_t kst, int64_t ksh, int64_t vst,
             int64_t vsh, uint4 *__restrict__ kc, uint8_t *__restrict__ ks, uint4 *__restrict__ vc,
             uint8_t *__restrict__ vs, Seqs s, int nb)
{
    pdl_wait();
    const int per_row = s.heads * nb;
    const int64_t total = int64_t(s.T) * 2 * per_row;
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    for (int64_t g = int64_t(blockIdx.x) * kThreads + threadIdx.x; g < total; g += stride) {
        const int t = int(g / (2 * per_row));
        int r = int(g - int64_t(t) * (2 * per_row));
        const bool is_v = r >= per_row;
        if (is_v) r -= per_row;
        const int h = r / nb, j = r - h * nb;
        const int b = seq_of_row(s, t);
        if (b < 0) continue;
        int lo, hi;
        seq_rows(s, b, lo, hi);
        const int64_t row = cache_row(s, b, h, int64_t(__ldg(s.len + b)) - hi + t);
        if (row < 0) continue;
        const int64_t off = int64_t(t) * (is_v ? vst : kst) + int64_t(h) * (is_v ? vsh : ksh) + 32 * j;
        float x[32];
        if constexpr (F32) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(is_v ? v : k) + off);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 a = __ldg(p + q);
                x[4 * q] = a.x;
                x[4 * q + 1] = a.y;
                x[4 * q + 2] = a.z;
                x[4 * q + 3] = a.w;
            }
        } else {
            uint4 raw[4];
            load_block(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(is_v ? v : k) + off), 0, raw);
            unpack32(raw, x);
        }
        uint4 c;
        uint32_t sb;
        mx_quantize_block(x, c, sb);
        (is_v ? vc : kc)[row * nb + j] = c;
        (is_v ? vs : ks)[row * nb + j] = uint8_t(sb);
    }
}

// Positions starts[b] + (row - cu[b]) of every sequence, decoded to bf16
// (exact but for overflow: two significant bits times a power of two) or
// fp32.  One thread per 32-block and array.  Rows that the table names no
// page for come out as zeros.
template <bool F32>
__global__ void __launch_bounds__(kThreads)
read_kernel(const uint4 *__restrict__ kc, const uint8_t *__restrict__ ks, const uint4 *__restrict__ vc,
            const uint8_t *__restrict__ vs, const int32_t *__restrict__ starts, void *__restrict__ out_k,
            void *__restrict__ out_v, Seqs s, int nb)
{
    pdl_wait();
    const int per_row = s.heads * nb;
    const int64_t total = int64_t(s.T) * 2 * per_row;
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    for (int64_t g = int64_t(blockIdx.x) * kThreads + threadIdx.x; g < total; g += stride) {
        const int t = int(g / (2 * per_row));
        int r = int(g - int64_t(t) * (2 * per_row));
        const bool is_v = r >= per_row;
        if (is_v) r -= per_row;
        const int h = r / nb, j = r - h * nb;
        const int b = seq_of_row(s, t);
        if (b < 0) continue;
        int lo, hi;
        seq_rows(s, b, lo, hi);
        const int64_t row = cache_row(s, b, h, int64_t(t - lo) + (starts ? __ldg(starts + b) : 0));
        uint4 c = make_uint4(0u, 0u, 0u, 0u);
        float sc = 0.0f;
        if (row >= 0) {
            c = __ldg((is_v ? vc : kc) + row * nb + j);
            sc = e8m0_value(__ldg((is_v ? vs : ks) + row * nb + j));
        }
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        const int64_t off = int64_t(t) * per_row + r;
        void *out = is_v ? out_v : out_k;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float2 e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[i] = e2m1x2_to_f32x2((w[q] >> (8 * i)) & 0xFFu);
                e[i].x *= sc;
                e[i].y *= sc;
            }
            if constexpr (F32) {
                float4 *o = static_cast<float4 *>(out) + off * 8 + 2 * q;
                o[0] = make_float4(e[0].x, e[0].y, e[1].x, e[1].y);
                o[1] = make_float4(e[2].x, e[2].y, e[3].x, e[3].y);
            } else {
                static_cast<uint4 *>(out)[off * 4 + q] =
                    make_uint4(mma::pack_bf16x2(e[0].x, e[0].y), mma::pack_bf16x2(e[1].x, e[1].y),
                               mma::pack_bf16x2(e[2].x, e[2].y), mma::pack_bf16x2(e[3].x, e[3].y));
            }
        }
    }
}

}  // namespace cache
