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
// to the sum with the block's two scales, in fp32:
//   sum[n][m] += (codes . x') * (2^(sb[n] - 127) * 2^ex[m])
// where x' = x 2^-ex is the block of x brought to fp16 by a power of two that
// puts its largest element in [2^14, 2^15): exact for bf16's 8 bits unless an
// element is below 2^-38 of the largest (then off by at most 2^-40 of it, the
// step of fp16's subnormals).  Blockwise, so that one loud channel costs no
// other block its bits.
//
// Layout.  A warp owns a tile of 16 weight rows: 4 consecutive lanes l of a
// 128-row scale group and their 4 quarters (rows base + 32 q + l), so that its
// scales of 128 channels are 64 consecutive bytes.  A stage is 256 channels:
// 16 rows x 128 bytes of codes and 2 x 64 of scales, brought by cp.async into
// the warp's own ring of kStages (nothing but the warp waits for it), the
// 16-byte pieces xor-swizzled by row, so that the 4-byte reads of 8 rows x 4
// words are conflict-free.  A CTA is 8 warps: RT row tiles x 8 / RT groups of
// channels; x is converted once per CTA for `kXBlocks` blocks at a time and
// shared by all warps.  The channels are also split over the CTAs of a
// cluster (up to 8), whose partial sums are added through distributed shared
// memory in rank order: one launch, no workspace, the same bits every time.

namespace gemv {

constexpr int kMaxRows = 32;
constexpr int kWarps = 8;
constexpr int kStages = 4;
constexpr int kChunkBlocks = 8;                               // 32-blocks per stage (256 channels)
constexpr int kCodeBytes = 16 * 16 * kChunkBlocks;            // 2048
constexpr int kScaleBytes = 16 * kChunkBlocks;                // 128
constexpr int kStageBytes = kCodeBytes + kScaleBytes;
constexpr int kTableBytes = 16 * kChunkBlocks * 4;            // decoded scales of the current stage
constexpr size_t kRing = size_t(kWarps) * (kStages * kStageBytes + kTableBytes);

// Blocks of x held at once: 32 KB of fp16 whatever the number of rows.
template <int NT>
constexpr int kXBlocks = 64 / NT;

template <int NT>
constexpr size_t kSmem = kRing + size_t(kXBlocks<NT>) * 8 * NT * (64 + 4);

// Copy 16 bytes if `full`, else write zeros (src is not read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool full)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
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

// A block of x as fp16 scaled by 2^-ex into dst (64 bytes); returns 2^ex.  The
// exponent is that of the largest finite element, so an infinity stays one
// and leaves the others their values.
__device__ __forceinline__ float x_block(const uint4 (&raw)[4], uint4 *dst)
{
    float v[32];
    unpack32(raw, v);
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float a = fabsf(v[i]);
        top = fmaxf(top, a <= 3.40282347e38f ? a : 0.0f);
    }
    // biased exponent of 2^ex: the largest element's less 14; at least 1 (2^-126:
    // bf16's subnormals are then multiples of 2^-7 and exact in fp16)
    const int field = max(int(__float_as_uint(top) >> 23) - 14, 1);
    const float down = __uint_as_float(uint32_t(254 - field) << 23);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        dst[q] = make_uint4(pack_f16x2(v[8 * q] * down, v[8 * q + 1] * down),
                            pack_f16x2(v[8 * q + 2] * down, v[8 * q + 3] * down),
                            pack_f16x2(v[8 * q + 4] * down, v[8 * q + 5] * down),
                            pack_f16x2(v[8 * q + 6] * down, v[8 * q + 7] * down));
    return __uint_as_float(uint32_t(field) << 23);
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
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
template <int RT, int NT, bool F32OUT>
__global__ void __launch_bounds__(kWarps * 32, NT == 4 ? 1 : 2)
mxf4_gemv_kernel(const __nv_bfloat16 *__restrict__ x, int64_t ldx, const uint8_t *__restrict__ codes,
                 const uint8_t *__restrict__ sf, void *__restrict__ out, int M, int N, int K, int S)
{
    pdl_wait();
    constexpr int KG = kWarps / RT;                           // channel groups
    constexpr int kLanes = 4 * RT;                            // lanes l of the scale group per CTA
    constexpr int XB = kXBlocks<NT>;
    constexpr int kRows = 16 * RT;
    static_assert(XB % (kChunkBlocks * KG) == 0, "a fill of x is whole rounds of the channel groups");
    extern __shared__ __align__(16) uint8_t smem_dyn[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane / 4, c = lane % 4;
    const int rt = warp % RT, kg = warp / RT;
    uint8_t *ring = smem_dyn + warp * (kStages * kStageBytes + kTableBytes);
    float4 *table = reinterpret_cast<float4 *>(ring + kStages * kStageBytes);
    uint4 *xs = reinterpret_cast<uint4 *>(smem_dyn + kRing);  // [XB][8 NT][64 bytes]
    float *xe = reinterpret_cast<float *>(smem_dyn + kRing + size_t(XB) * 8 * NT * 64);   // [XB][8 NT]

    const int part = int(blockIdx.x) / S, rank = int(blockIdx.x) % S;
    const int group = part / KG, l0 = (part % KG) * kLanes + 4 * rt;       // the warp's lanes: l0 .. l0 + 3
    const int nb = K / 32, Ka = (nb + 3) / 4, KC = (nb + kChunkBlocks - 1) / kChunkBlocks;
    const int c0 = int(int64_t(rank) * KC / S), c1 = int(int64_t(rank + 1) * KC / S);

    // this lane's pieces of a stage: rows (lane / 8) + 4 j (= lane l0 + lane / 8, quarter j), piece lane % 8
    const int piece = lane % 8;
    const int n0 = group * 128 + l0 + lane / 8;
    const uint8_t *src = codes + int64_t(n0) * (K / 2) + piece * 16;
    const uint8_t *ssrc = sf + int64_t(group) * Ka * 512 + (lane / 4) * 512 + l0 * 16 + (lane % 4) * 16;
    const uint32_t ring_s = smem_addr(ring);

    // stage `slot` <- chunk ch (or nothing past the rank's last)
    auto fetch = [&](int ch, int slot) {
        if (ch < c1) {
            const uint32_t dst = ring_s + slot * kStageBytes;
            const bool in_k = ch * kChunkBlocks + piece < nb;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = 4 * j + lane / 8;
                const bool full = in_k && n0 + 32 * j < N;
                cp_async16_or_zero(dst + row * 128 + ((piece ^ (row & 7)) << 4),
                                   full ? src + int64_t(32 * j) * (K / 2) + int64_t(ch) * 128 : codes, full);
            }
            if (lane < 8) {
                const bool full = 2 * ch + lane / 4 < Ka;
                cp_async16_or_zero(dst + kCodeBytes + lane * 16, full ? ssrc + int64_t(ch) * 1024 : sf, full);
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
    for (int i = 0; i < kStages - 1; ++i) fetch(c0 + i * KG + kg, i);
    int it = 0;
    for (int f0 = c0; f0 < c1; f0 += XB / kChunkBlocks) {
        // ---- x of the next XB blocks: fp16 and the powers of two
        __syncthreads();
        const int blocks = min(XB, nb - f0 * kChunkBlocks);
        for (int i = threadIdx.x; i < XB * 8 * NT; i += kWarps * 32) {
            const int j = i % XB, m = i / XB;                 // consecutive threads: consecutive blocks of a row
            uint4 *dst = xs + (j * 8 * NT + m) * 4;
            float s = 0.0f;
            if (m < M && j < blocks) {
                uint4 raw[4];
                load_block(reinterpret_cast<const uint4 *>(x + m * ldx + int64_t(f0 * kChunkBlocks + j) * 32), 0, raw);
                s = x_block(raw, dst);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) dst[q] = make_uint4(0u, 0u, 0u, 0u);
            }
            xe[j * 8 * NT + m] = s;
        }
        __syncthreads();
        const int f1 = min(c1, f0 + XB / kChunkBlocks);
        for (int ch = f0 + kg; ch < f1; ch += KG, ++it) {
            cp_wait<kStages - 2>();
            __syncwarp();
            fetch(ch + (kStages - 1) * KG, (it + kStages - 1) % kStages);
            const uint8_t *st = ring + (it % kStages) * kStageBytes;
            {
                // the stage's 128 scales as floats, [unit][row][4]: lane = unit * 16 + (l * 4 + quarter)
                const uint32_t w = reinterpret_cast<const uint32_t *>(st + kCodeBytes)[lane];
                const int blk = ch * kChunkBlocks + (lane / 16) * 4;
                float4 s;
                s.x = blk < nb ? e8m0_value(w & 0xFFu) : 0.0f;
                s.y = blk + 1 < nb ? e8m0_value((w >> 8) & 0xFFu) : 0.0f;
                s.z = blk + 2 < nb ? e8m0_value((w >> 16) & 0xFFu) : 0.0f;
                s.w = blk + 3 < nb ? e8m0_value(w >> 24) : 0.0f;
                table[(lane & 16) + (lane & 3) * 4 + ((lane >> 2) & 3)] = s;
            }
            __syncwarp();
            const uint4 *xc = xs + ((ch - f0) * kChunkBlocks * 8 * NT + g) * 4 + c;
            const float *xf = xe + (ch - f0) * kChunkBlocks * 8 * NT + 2 * c;
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
                        const uint4 bx = xc[(j * NT + t) * 32];
                        const float2 e = *reinterpret_cast<const float2 *>(xf + (j * NT + t) * 8);
                        float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma_f16(p, a[0], d[0], a[1], d[1], bx.x, bx.y);
                        mma_f16(p, a[2], d[2], a[3], d[3], bx.z, bx.w);
                        acc[t][0] = fmaf(p[0], lo[b] * e.x, acc[t][0]);
                        acc[t][1] = fmaf(p[1], lo[b] * e.y, acc[t][1]);
                        acc[t][2] = fmaf(p[2], hi[b] * e.x, acc[t][2]);
                        acc[t][3] = fmaf(p[3], hi[b] * e.y, acc[t][3]);
                    }
                }
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
