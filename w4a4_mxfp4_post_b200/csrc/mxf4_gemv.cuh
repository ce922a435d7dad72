// mxf4_gemv.cuh -- a few rows times MXFP4 weights.  Included by kroquant.cu;
// uses its helpers.
//
//   out[m][n] = sum_k x[m][k] b[n][k],   M <= 32
//
// x is bf16 and not quantized; b is the weight operand of mxf4_gemm (codes
// [N][K/2], scales in the scale-factor layout), so one copy of the weights
// serves both products.

namespace gemv {

constexpr int kMaxRows = 32;

// One warp per weight row and activation row.
template <bool F32OUT>
__global__ void __launch_bounds__(kThreads)
rows_kernel(const __nv_bfloat16 *__restrict__ x, int64_t ldx, const uint8_t *__restrict__ codes,
            const uint8_t *__restrict__ sf, void *__restrict__ out, int M, int64_t N, int K)
{
    pdl_wait();
    const int lane = threadIdx.x % 32;
    const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / 32;
    if (w >= N * M) return;
    const int64_t n = w / M;
    const int m = int(w % M);
    const int nb = K / 32;
    float acc = 0.0f;
    for (int j = lane; j < nb; j += 32) {
        const int64_t unit = (n / 128) * ((nb + 3) / 4) + j / 4;
        const float s = e8m0_value(sf[unit * 512 + (n % 32) * 16 + (n / 32 % 4) * 4 + j % 4]);
        float blk = 0.0f;
        for (int i = 0; i < 16; ++i) {
            const float2 e = e2m1x2_to_f32x2(codes[n * (K / 2) + 16 * j + i]);
            blk = fmaf(__bfloat162float(x[m * ldx + 32 * j + 2 * i]), e.x, blk);
            blk = fmaf(__bfloat162float(x[m * ldx + 32 * j + 2 * i + 1]), e.y, blk);
        }
        acc = fmaf(blk, s, acc);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
    if (lane == 0) {
        if constexpr (F32OUT) static_cast<float *>(out)[m * N + n] = acc;
        else static_cast<__nv_bfloat16 *>(out)[m * N + n] = __float2bfloat16_rn(acc);
    }
}

}  // namespace gemv
