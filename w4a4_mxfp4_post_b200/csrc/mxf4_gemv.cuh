// mxf4_gemv.cuh -- a few rows times MXFP4 weights.  Included by kroquant.cu;
// uses its helpers.
//
//   out[m][n] = sum_k x[m][k] b[n][k],   M <= 32
//
// x is bf16 and not quantized; b is the weight operand of mxf4_gemm (codes
// [N][K/2], scales in the scale-factor layout), so one copy of the weights
// serves both products.
//
// Bound: the weights are read once, 17/32 byte per element, and used for M
// products each, so the kernel lives off HBM; what it must not do is spend
// more issue slots than the bytes leave it.  At 6.5 TB/s an SM sub-partition
// gets 5.8 bytes per clock, 11 weights.  So the weights go through the tensor
// cores as fp16 codes: cvt.rn.f16x2.e2m1x2 unpacks two per instruction (2
// clocks measured; the shift-and-mask expansion to bf16 took 6.4 per pair),
// unscaled, as the 16-row operand of mma.m16n8k16, and x is the 8-column one.
// (The legacy MMA is enough: 8 clocks for 16 x 16 weights, a quarter of what
// their bytes take; a tcgen05 MMA would need the codes in shared memory.)
// The two MMAs of a 32-block run into a zero accumulator, which is then added
// to the chunk's sum with the block's scale, and the chunk's to the whole, in
// fp32:
//   chunk[n][m] += (codes . x') * 2^(sb[n] - 127),   sum[n][m] += chunk[n][m] * 2^ex[m]
// where x' = x 2^-ex is a chunk (256 channels) of x brought to fp16 by a power
// of two that puts its largest element in [2^15, 2^16): bf16's 8 bits stay
// exact down to 2^-32 of the largest; what is below is off by at most 2^-40 of
// it, half the step of fp16's subnormals.  (Where a scale is 2^97 or more, 2^ex comes first.)
//
// Layout.  A warp owns a tile of 16 weight rows: 4 consecutive lanes l of a
// 128-row scale group and their 4 quarters (rows base + 32 q + l), so that its
// scales of 128 channels are 64 consecutive bytes.  A stage is 256 channels:
// 16 rows x 128 bytes of codes and 2 x 64 of scales, brought by cp.async into
// the warp's own ring (nothing but the warp waits for it), the
// 16-byte pieces xor-swizzled by row, so that the 4-byte reads of 8 rows x 4
// words are conflict-free.  A CTA is 8 warps: RT row tiles x 8 / RT groups of
// channels; x is converted once per CTA for `kXChunks` chunks at a time and
// shared by all warps.  Where that conversion is a good part of the work (many
// rows, or many CTAs converting the same x) a kernel of its own does it once, in
// the layout that the product reads, and x comes by cp.async with the weights,
// the chunks of a stage for all of the CTA's warps (PRE).  The channels are also
// split over the CTAs of a cluster (up to 8), whose partial sums are added
// through distributed shared memory in rank order: the same bits every time.
//
// Measured, 8192 x 28672 weights (125 MB; a cp.async loop that only reads them
// takes 28 to 31 us): 1 row 33 us, 3.7 TB/s; 8 rows 37; 16 rows 50 (63 with x
// converted in every CTA); 32 rows 76.  With 16 rows issue slots are 45 % and the
// tensor pipe 31 % busy, 3.4 warps to a scheduler: shared-memory reads of x (16
// bytes for every 4 of codes) and the barrier per stage are in the way.  Small
// products whose x is converted in every CTA convert more of it than they use:
// a rank of 5 x 5600 x 2240 takes 2 or 3 of the 9 chunks and converts up to 8 (9 us,
// of which a launch is 3).

namespace gemv {

constexpr int kMaxRows = 32;
constexpr int kWarps = 8;
template <int NT>
constexpr int kStages = NT == 4 ? 3 : 4;                      // (3: two CTAs of 32 rows fit on an SM, 32 x 4096 x 4096 24 -> 13 us)
constexpr int kChunkBlocks = 8;                               // 32-blocks per stage (256 channels)
constexpr int kCodeBytes = 16 * 16 * kChunkBlocks;            // 2048
constexpr int kScaleBytes = 16 * kChunkBlocks;                // 128
constexpr int kStageBytes = kCodeBytes + kScaleBytes;
constexpr int kTableBytes = 16 * kChunkBlocks * 4;            // decoded scales of the current stage
template <int NT>
constexpr size_t kRing = size_t(kWarps) * (kStages<NT> * kStageBytes + kTableBytes);

// Chunks of x held at once: 32 KB of fp16 whatever the number of rows.  A
// block's rows are 64 bytes each, and 64 bytes of padding put two consecutive
// blocks of a row into different halves of the banks.
template <int NT>
constexpr int kXChunks = 8 / NT;
template <int NT>
constexpr int kXBlockBytes = 8 * NT * 64 + 64;
template <int NT>
constexpr int kXBytes = kXChunks<NT> * kChunkBlocks * kXBlockBytes<NT>;

template <int NT>
constexpr int kXStage = kChunkBlocks * kXBlockBytes<NT> + 8 * NT * 4;                    // PRE: a chunk and its exponents

template <int RT, int NT, bool PRE>
constexpr size_t kSmem = kRing<NT> + (PRE ? size_t(kStages<NT>) * kXStage<NT> * (kWarps / RT)
                                          : size_t(kXBytes<NT>) + size_t(kXChunks<NT>) * 8 * NT * 4);

// x converted beforehand: [K / 32, whole chunks][rows, 8 NT][32] fp16, then
// [chunks][rows] fp32 exponents.
__host__ __device__ constexpr int64_t x_elements(int64_t KC, int rows) { return KC * kChunkBlocks * rows * 32; }
__host__ __device__ constexpr int64_t x_bytes(int64_t KC, int rows) { return x_elements(KC, rows) * 2 + KC * rows * 4; }

// Copy `bytes` (16, or 0: src is not read) and fill up 16 bytes with zeros.
__device__ __forceinline__ void cp_async16_sized(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight codes of a word as four f16 pairs, in order.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 q0, q1, q2, q3;\n\t"
        "mov.b32 {q0, q1, q2, q3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, q0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, q1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, q2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, q3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// c += A B, A 16 x 16 (row), B 16 x 8 (col), f16 with fp32 sums.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 elements of a chunk of x (the warp holds its 256) as fp16 scaled by 2^-ex;
// e = 2^ex.  The exponent is that of the largest finite element, so an
// infinity stays one and leaves the others their values.
__device__ __forceinline__ uint4 x_chunk(const uint4 raw, float &e)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    // magnitudes as 16-bit patterns, which order like the numbers
    uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    top = __reduce_max_sync(0xffffffffu, max(top << 16, top & 0xffff0000u));
    if (top >= 0x7f800000u) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = (w[i] << 16) & 0x7fff0000u, hi = w[i] & 0x7fff0000u;
            top = max(top, max(lo < 0x7f800000u ? lo : 0u, hi < 0x7f800000u ? hi : 0u));
        }
        top = __reduce_max_sync(0xffffffffu, top);
    }
    // biased exponent of 2^ex: the largest element's less 15; at least 1 (2^-126:
    // bf16's subnormals are then multiples of 2^-7 and exact in fp16)
    const int field = max(int(top >> 23) - 15, 1);
    const float down = __uint_as_float(uint32_t(254 - field) << 23);
    e = __uint_as_float(uint32_t(field) << 23);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = pack_f16x2(bf16_lo(w[i]) * down, bf16_hi(w[i]) * down);
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// Four scale bytes as their values: the byte is the exponent field of 2^(byte -
// 127), but for 0 (the subnormal 2^-127) and 255 (NaN).
__device__ __forceinline__ float4 scales4(uint32_t w)
{
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = max(__byte_perm(w, 0, 0x0444 | (i << 12)) >> 1, 0x00400000u);
    if ((~w - 0x01010101u) & w & 0x80808080u) {               // some byte is 255
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] |= v[i] == 0x7f800000u ? 0x00400000u : 0u;
    }
    return make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
}

// A warp per row and chunk; rows M .. rows - 1 are zeros.
__global__ void __launch_bounds__(256)
convert_kernel(const __nv_bfloat16 *__restrict__ x, int64_t ldx, uint8_t *__restrict__ xw, int M, int rows, int nb, int KC)
{
    pdl_wait();
    const int lane = threadIdx.x % 32;
    const int64_t i = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
    if (i >= int64_t(KC) * rows) return;
    const int m = int(i % rows), ch = int(i / rows), blk = ch * kChunkBlocks + lane / 4;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (m < M && blk < nb) raw = __ldg(reinterpret_cast<const uint4 *>(x + m * ldx + int64_t(blk) * 32 + (lane % 4) * 8));
    float e;
    const uint4 h = x_chunk(raw, e);
    reinterpret_cast<uint4 *>(xw)[(int64_t(blk) * rows + m) * 4 + lane % 4] = h;
    if (lane == 0) reinterpret_cast<float *>(xw + x_elements(KC, rows) * 2)[int64_t(ch) * rows + m] = m < M ? e : 0.0f;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A float of the same shared-memory variable in CTA `rank` of the cluster.
__device__ __forceinline__ float cluster_load(const float *p, uint32_t rank)
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Grid: (8 / RT parts of every 128-row group) x S ranks, rank fastest (a
// cluster is the S ranks of one part).  Rank r takes chunks [r KC / S,
// (r + 1) KC / S) of the KC = ceil(K / 256), in turn by the CTA's channel groups.
template <int RT, int NT, bool PRE, bool F32OUT>
__global__ void __launch_bounds__(kWarps * 32, 2)
mxf4_gemv_kernel(const __nv_bfloat16 *__restrict__ x, int64_t ldx, const uint8_t *__restrict__ codes,
                 const uint8_t *__restrict__ sf, const uint8_t *__restrict__ xw, void *__restrict__ out, int M, int N, int K,
                 int S)
{
    pdl_wait();
    constexpr int KG = kWarps / RT;                           // channel groups
    constexpr int kLanes = 4 * RT;                            // lanes l of the scale group per CTA
    constexpr int XC = kXChunks<NT>;
    constexpr int kRows = 16 * RT;
    constexpr int ST = kStages<NT>;
    static_assert(PRE || XC % KG == 0, "a fill of x is whole rounds of the channel groups");
    extern __shared__ __align__(16) uint8_t smem_dyn[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane / 4, c = lane % 4;
    const int rt = warp % RT, kg = warp / RT;
    uint8_t *ring = smem_dyn + warp * (ST * kStageBytes + kTableBytes);
    float4 *table = reinterpret_cast<float4 *>(ring + ST * kStageBytes);
    uint8_t *xs = smem_dyn + kRing<NT>;                         // [blocks][8 NT rows of 64 bytes, padding]
    float *xe = reinterpret_cast<float *>(xs + kXBytes<NT>);  // [XC][8 NT] (both: not with PRE)

    const int part = int(blockIdx.x) / S, rank = int(blockIdx.x) % S;
    const int group = part / KG, l0 = (part % KG) * kLanes + 4 * rt;       // the warp's lanes: l0 .. l0 + 3
    const int nb = K / 32, Ka = (nb + 3) / 4, KC = (nb + kChunkBlocks - 1) / kChunkBlocks;
    const int c0 = int(int64_t(rank) * KC / S), c1 = int(int64_t(rank + 1) * KC / S);

    // this lane's pieces of a stage: rows (lane / 8) + 4 j (lane l0 + lane / 8 of
    // the group, quarter j), piece lane % 8; rows past N are zeros
    const int piece = lane % 8;
    const int n0 = group * 128 + l0 + lane / 8;
    const uint8_t *src[4];
    uint32_t size[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        size[j] = n0 + 32 * j < N ? 16 : 0;
        src[j] = codes + int64_t(min(n0 + 32 * j, N - 1)) * (K / 2) + int64_t(c0 + kg) * 128 + piece * 16;
    }
    const uint8_t *ssrc = sf + (int64_t(group) * Ka + 2 * (c0 + kg) + (lane / 4) % 2) * 512 + l0 * 16 + (lane % 4) * 16;
    const uint32_t ring_s = smem_addr(ring);
    const uint32_t dst0 = ring_s + (lane / 8) * 128 + ((piece ^ (lane / 8)) << 4);
    const uint32_t dst1 = ring_s + (lane / 8) * 128 + ((piece ^ (lane / 8 + 4)) << 4);

    // stage `slot` <- chunk ch, the warp's next (or nothing past the rank's last)
    auto fetch = [&](int ch, int slot) {
        if (ch < c1) {
            const uint32_t at = slot * kStageBytes;
            const bool in_k = ch * kChunkBlocks + piece < nb;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cp_async16_sized((j % 2 ? dst1 : dst0) + at + j * 512, in_k ? src[j] : codes, in_k ? size[j] : 0);
                src[j] += KG * 128;
            }
            if (lane < 8) {
                const bool in_a = 2 * ch + lane / 4 < Ka;
                cp_async16_sized(ring_s + at + kCodeBytes + lane * 16, in_a ? ssrc : sf, in_a ? 16 : 0);
            }
            ssrc += KG * 1024;
        }
        if constexpr (PRE) {                                  // the CTA's threads bring the chunks of x together
#pragma unroll
            for (int kk = 0; kk < KG; ++kk) {
                const int cx = ch - kg + kk;
                if (cx >= c1) break;
                const uint32_t to = smem_addr(xs) + (slot * KG + kk) * kXStage<NT>;
                const uint8_t *from = xw + int64_t(cx) * kChunkBlocks * 8 * NT * 64;
#pragma unroll
                for (int j = 0; j < NT; ++j) {                // 256 NT pieces, 32 NT to a block
                    const int i = threadIdx.x + 256 * j;
                    cp_async16_sized(to + i / (32 * NT) * kXBlockBytes<NT> + i % (32 * NT) * 16, from + i * 16, 16);
                }
                if (threadIdx.x < 2 * NT)
                    cp_async16_sized(to + kChunkBlocks * kXBlockBytes<NT> + threadIdx.x * 16,
                                     xw + x_elements(KC, 8 * NT) * 2 + int64_t(cx) * 8 * NT * 4 + threadIdx.x * 16, 16);
            }
        }
        cp_commit();
    };

    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;

#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(c0 + i * KG + kg, i);
    const bool row_there = group * 128 + (lane & 3) * 32 + l0 + ((lane >> 2) & 3) < N;    // of this lane's scale bytes
    // chunk ch of the stage at `st` times x at `xc` with the exponents `ex`
    auto product = [&](int ch, const uint8_t *st, const uint8_t *xc, const float *ex) {
        bool large;                                           // some scale is 2^97 or more (or NaN)
        {
            // the stage's 128 scales as floats, [unit][row][4]: lane = unit * 16 + (l * 4 + quarter)
            const uint32_t w = reinterpret_cast<const uint32_t *>(st + kCodeBytes)[lane];
            float4 s = scales4(w);
            large = __any_sync(0xffffffffu, row_there && (w & (w << 1) & (w << 2) & 0x80808080u) != 0);
            const int left = nb - (ch * kChunkBlocks + (lane / 16) * 4);
            if (left < 4) {                               // padding bytes of the last unit may hold anything
                if (left < 1) s.x = 0.0f;
                if (left < 2) s.y = 0.0f;
                if (left < 3) s.z = 0.0f;
                s.w = 0.0f;
            }
            table[(lane & 16) + (lane & 3) * 4 + ((lane >> 2) & 3)] = s;
        }
        __syncwarp();
        xc += g * 64 + c * 16;
        if (large) {
            // x' carries up to 2^16 and a block's sum 2^24: times such a scale that may pass fp32's range although the
            // product does not.  The exponent of x is applied first then, block by block (last where the scale is
            // below 1, for the same reason).  Rare: not unrolled.
#pragma unroll 1
            for (int j = 0; j < kChunkBlocks; ++j) {
                const uint8_t *row = st + g * 128 + ((j ^ g) << 4) + c * 4;
                const float *scale = reinterpret_cast<const float *>(table + (j / 4) * 16 + g) + j % 4;
                const float lo = scale[0], hi = scale[8 * 4];
                uint32_t a[4], d[4];
                codes_f16(*reinterpret_cast<const uint32_t *>(row), a);
                codes_f16(*reinterpret_cast<const uint32_t *>(row + 8 * 128), d);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 bx = *reinterpret_cast<const uint4 *>(xc + j * kXBlockBytes<NT> + t * 512);
                    const float2 e = *reinterpret_cast<const float2 *>(ex + 8 * t + 2 * c);
                    float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_f16(p, a[0], d[0], a[1], d[1], bx.x, bx.y);
                    mma_f16(p, a[2], d[2], a[3], d[3], bx.z, bx.w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float f = i < 2 ? lo : hi, ei = i % 2 ? e.y : e.x;
                        acc[t][i] = f >= 1.0f ? fmaf(p[i] * ei, f, acc[t][i]) : fmaf(p[i] * f, ei, acc[t][i]);
                    }
                }
            }
            return;
        }
        float sum[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[t][i] = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float4 t0 = table[u * 16 + g], t1 = table[u * 16 + g + 8];
            const float lo[4] = {t0.x, t0.y, t0.z, t0.w}, hi[4] = {t1.x, t1.y, t1.z, t1.w};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int j = 4 * u + b;
                const uint8_t *row = st + g * 128 + ((j ^ g) << 4) + c * 4;
                uint32_t a[4], d[4];
                codes_f16(*reinterpret_cast<const uint32_t *>(row), a);
                codes_f16(*reinterpret_cast<const uint32_t *>(row + 8 * 128), d);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 bx = *reinterpret_cast<const uint4 *>(xc + j * kXBlockBytes<NT> + t * 512);
                    float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_f16(p, a[0], d[0], a[1], d[1], bx.x, bx.y);
                    mma_f16(p, a[2], d[2], a[3], d[3], bx.z, bx.w);
                    sum[t][0] = fmaf(p[0], lo[b], sum[t][0]);
                    sum[t][1] = fmaf(p[1], lo[b], sum[t][1]);
                    sum[t][2] = fmaf(p[2], hi[b], sum[t][2]);
                    sum[t][3] = fmaf(p[3], hi[b], sum[t][3]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float2 e = *reinterpret_cast<const float2 *>(ex + 8 * t + 2 * c);
            acc[t][0] = fmaf(sum[t][0], e.x, acc[t][0]);
            acc[t][1] = fmaf(sum[t][1], e.y, acc[t][1]);
            acc[t][2] = fmaf(sum[t][2], e.x, acc[t][2]);
            acc[t][3] = fmaf(sum[t][3], e.y, acc[t][3]);
        }
    };
    if constexpr (PRE) {
        for (int ch = c0 + kg, it = 0; ch - kg < c1; ch += KG, ++it) {
            cp_wait<ST - 2>();
            __syncthreads();                                  // everybody's pieces are there, the stage before is free
            fetch(ch + (ST - 1) * KG, (it + ST - 1) % ST);
            const uint8_t *xc = xs + (it % ST * KG + kg) * kXStage<NT>;
            if (ch < c1)
                product(ch, ring + (it % ST) * kStageBytes, xc, reinterpret_cast<const float *>(xc + kChunkBlocks * kXBlockBytes<NT>));
        }
    } else {
        // columns of no row stay zero
        for (int i = threadIdx.x; i < XC * kChunkBlocks * 8 * NT * 4; i += kWarps * 32) {
            const int m = i / 4 % (8 * NT), j = i / (32 * NT);
            if (m >= M) *reinterpret_cast<uint4 *>(xs + j * kXBlockBytes<NT> + m * 64 + (i % 4) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (threadIdx.x < XC * 8 * NT) xe[threadIdx.x] = 0.0f;
        int it = 0;
        for (int f0 = c0; f0 < c1; f0 += XC) {
            // ---- the next XC chunks of x, a row's chunk per warp and turn
            __syncthreads();
#pragma unroll 4
            for (int i = warp; i < XC * M; i += kWarps) {
                const int cc = i % XC, m = i / XC, blk = (f0 + cc) * kChunkBlocks + lane / 4;
                if ((f0 + cc) * kChunkBlocks >= nb) continue;
                uint4 raw = make_uint4(0u, 0u, 0u, 0u);
                if (blk < nb)
                    raw = __ldg(reinterpret_cast<const uint4 *>(x + m * ldx + int64_t(blk) * 32 + (lane % 4) * 8));
                float e;
                const uint4 h = x_chunk(raw, e);
                *reinterpret_cast<uint4 *>(xs + (cc * kChunkBlocks + lane / 4) * kXBlockBytes<NT> + m * 64 + (lane % 4) * 16) = h;
                if (lane == 0) xe[cc * 8 * NT + m] = e;
            }
            __syncthreads();
            const int f1 = min(c1, f0 + XC);
            for (int ch = f0 + kg; ch < f1; ch += KG, ++it) {
                cp_wait<ST - 2>();
                __syncwarp();
                fetch(ch + (ST - 1) * KG, (it + ST - 1) % ST);
                product(ch, ring + (it % ST) * kStageBytes, xs + (ch - f0) * kChunkBlocks * kXBlockBytes<NT>, xe + (ch - f0) * 8 * NT);
            }
        }
    }
    cp_wait<0>();
    __syncthreads();

    // ---- sums over the channel groups and the cluster's ranks, in that order.
    // red[kg][m][quarter * kLanes + lane]: the rows of one quarter are consecutive.
    float *red = reinterpret_cast<float *>(smem_dyn);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = g + 8 * (i >> 1), m = 8 * t + 2 * c + (i & 1);
            red[(kg * 8 * NT + m) * kRows + (row >> 2) * kLanes + 4 * rt + (row & 3)] = acc[t][i];
        }
    if (S > 1) cluster_sync();
    else __syncthreads();
    const int total = M * kRows;
    const int e0 = int(int64_t(rank) * total / S), e1 = int(int64_t(rank + 1) * total / S);
    for (int e = e0 + threadIdx.x; e < e1; e += kWarps * 32) {
        const int m = e / kRows, slot = e % kRows;
        float v = 0.0f;
        for (int r = 0; r < S; ++r) {
#pragma unroll
            for (int k = 0; k < KG; ++k) {
                const float *p = red + (k * 8 * NT + m) * kRows + slot;
                v += S > 1 ? cluster_load(p, r) : *p;
            }
        }
        const int n = group * 128 + (slot / kLanes) * 32 + (part % KG) * kLanes + slot % kLanes;
        if (n < N) {
            if constexpr (F32OUT) static_cast<float *>(out)[int64_t(m) * N + n] = v;
            else static_cast<__nv_bfloat16 *>(out)[int64_t(m) * N + n] = __float2bfloat16_rn(v);
        }
    }
    if (S > 1) cluster_sync();                                // nobody leaves while its sums are read
}

}  // namespace gemv
