// mx_attention.cuh -- attention of a chunk of new tokens over a paged MXFP4
// cache.  Included by kroquant.cu; uses its helpers and mx_cache.cuh.
//
//   out[t][h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[t][h] . k_j - max)
//
// over the positions j of t's sequence that its mask leaves: j <= the
// position of t (causal) or every j below the sequence's length.  Positions
// whose page the table does not name are not seen.  A row that sees nothing
// is zero.

namespace attn {

struct Args {
    const __nv_bfloat16 *q;
    int64_t q_st, q_sh;                      // strides of a token and a head (elements)
    const uint8_t *kc, *ks, *vc, *vs;
    __nv_bfloat16 *out;                      // [T][hq][D]
    float scale_log2;                        // scale * log2(e)
    int causal;
    int hq, group;                           // query heads, query heads per kv head
    cache::Seqs s;
};

// The value of a scale byte; 253 to 255 read as NaN (a code of 4 or 6 would
// pass fp32's range with the first two).
__device__ __forceinline__ float scale_value(uint32_t sb) { return e8m0_value(sb >= 253u ? 255u : sb); }

// One warp per (token, query head): lanes hold D / 32 channels each.
template <int D>
__global__ void __launch_bounds__(kThreads)
rows_kernel(Args a)
{
    pdl_wait();
    constexpr int C = D / 32;                // channels per lane
    const int lane = threadIdx.x % 32;
    const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / 32;
    if (w >= int64_t(a.s.T) * a.hq) return;
    const int t = int(w / a.hq), h = int(w % a.hq), kvh = h / a.group;
    const int b = cache::seq_of_row(a.s, t);
    if (b < 0) return;
    int lo, hi;
    cache::seq_rows(a.s, b, lo, hi);
    const int len = __ldg(a.s.len + b);
    int64_t end = a.causal ? int64_t(len) - hi + t + 1 : len;
    end = min(end, cache::seq_cap(a.s));
    float qv[C], o[C];
    const int ch0 = lane * C;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        qv[i] = __bfloat162float(a.q[int64_t(t) * a.q_st + int64_t(h) * a.q_sh + ch0 + i]);
        o[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = 0; j < end; ++j) {
        const int64_t row = cache::cache_row(a.s, b, kvh, j);
        if (row < 0) continue;
        float s = 0.0f, v[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int ch = ch0 + i;
            const int64_t at = row * (D / 2) + ch / 2, sat = row * (D / 32) + ch / 32;
            const float2 kk = e2m1x2_to_f32x2(a.kc[at]), vv = e2m1x2_to_f32x2(a.vc[at]);
            s = fmaf(qv[i], ((ch & 1) ? kk.y : kk.x) * scale_value(a.ks[sat]), s);
            v[i] = ((ch & 1) ? vv.y : vv.x) * scale_value(a.vs[sat]);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale_log2;
        const float mn = s > m || s != s ? s : m;
        const float r = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = fmaf(l, r, p);
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = fmaf(o[i], r, p * v[i]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < C; ++i)
        a.out[(int64_t(t) * a.hq + h) * D + ch0 + i] = __float2bfloat16_rn(l == 0.0f ? 0.0f : o[i] * inv);
}

}  // namespace attn
