// kv4_attention.cu -- softmax attention over the 4-bit paged KV cache.
//
// Method: bitnet_v2_engine.py page, BitNetV2Attention.forward on the fake-quantised keys and
// values: s_t = scale * kstep_t * (q . kcode_t), out = sum_t e^(s_t) vstep_t vcode_t / sum_t e^(s_t).
//
// One CTA per (row, query head); each warp takes every fourth position with a running maximum,
// sum and output, and the four are joined at the end.
#include "kv4.cuh"

#include <math_constants.h>

namespace bitnet {

namespace {

constexpr int kWarps = 4;

template <bool BF16>
__device__ __forceinline__ float load1(const void *x, int64_t i) {
    if constexpr (BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(x)[i]);
    else return reinterpret_cast<const float *>(x)[i];
}

// The lane's E = D / 32 codes of a row.
template <int E>
__device__ __forceinline__ void codes_of(const uint8_t *row, int lane, float *y) {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
        const int b = row[lane * (E / 2) + j];
        y[2 * j] = (float)((int)(b << 28) >> 28);
        y[2 * j + 1] = (float)((int)(b << 24) >> 28);
    }
}

template <bool BF16, int D>
__global__ void __launch_bounds__(32 * kWarps)
kv4_attention_kernel(const void *__restrict__ q, int64_t qts, int64_t qhs, int q_heads, Kv4Cache c, Kv4Batch bt,
                     float scale, int causal, int64_t window, void *__restrict__ out, float *__restrict__ lse,
                     int *status) {
    constexpr int E = D / 32;
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int t = blockIdx.x, h = blockIdx.y, kh = h / (q_heads / c.heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int b, pos;
    if (!kv4_locate(bt, t, b, pos)) return;
    const int len = __ldg(bt.lens + b);
    const int end = causal ? min(len, pos + 1) : len;
    const int begin = (causal && window > 0) ? (int)max((int64_t)0, (int64_t)pos - window + 1) : 0;
    float qv[E], o[E], m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = load1<BF16>(q, t * qts + h * qhs + lane * E + e);
        o[e] = 0.0f;
    }
    for (int s = begin + warp; s < end; s += kWarps) {
        const int page = kv4_page(c, bt, b, s, status);
        if (page < 0) continue;
        const int64_t row = kv4_rows(c, page, kh) + (s & ((1 << c.page_log2) - 1));
        float kc[E], vc[E];
        if (s == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                kc[e] = (float)c.k_bos[((int64_t)page * c.heads + kh) * D + lane * E + e];
                vc[e] = (float)c.v_bos[((int64_t)page * c.heads + kh) * D + lane * E + e];
            }
        } else {
            codes_of<E>(c.k_codes + row * (D / 2), lane, kc);
            codes_of<E>(c.v_codes + row * (D / 2), lane, vc);
        }
        float z = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) z = fmaf(qv[e], kc[e], z);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
        z *= c.k_step[row] * scale;
        const float m2 = fmaxf(m, z);
        const float a = m == -CUDART_INF_F ? 0.0f : expf(m - m2), w = expf(z - m2);
        const float wv = w * c.v_step[row];
        l = fmaf(l, a, w);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], a, wv * vc[e]);
        m = m2;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    __syncthreads();
    float top = -CUDART_INF_F, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
    float f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        f[w] = sm[w] == -CUDART_INF_F ? 0.0f : expf(sm[w] - top);
        sum += f[w] * sl[w];
    }
    const int64_t base = ((int64_t)t * q_heads + h) * D;
    for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) y += f[w] * so[w][d];
        y = sum > 0.0f || sum != sum ? y / sum : 0.0f;
        if constexpr (BF16) reinterpret_cast<__nv_bfloat16 *>(out)[base + d] = __float2bfloat16_rn(y);
        else reinterpret_cast<float *>(out)[base + d] = y;
    }
    if (lse && threadIdx.x == 0) lse[(int64_t)t * q_heads + h] = sum > 0.0f || sum != sum ? top + logf(sum) : -CUDART_INF_F;
}

}  // namespace

size_t kv4_attention_workspace(int64_t, int, int, int, int) { return 256; }

cudaError_t launch_kv4_attention(const void *q, bool bf16, int64_t T, int q_heads, int64_t qts, int64_t qhs,
                                 const Kv4Cache &c, const Kv4Batch &bt, float scale, bool causal, int64_t window,
                                 int64_t, void *out, float *lse, void *, cudaStream_t s) {
    auto go = [&](auto kernel) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)T, (unsigned)q_heads);
        cfg.blockDim = dim3(32 * kWarps);
        cfg.stream = s;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kernel, q, qts, qhs, q_heads, c, bt, scale, (int)causal, window, out, lse,
                                  device_status_ptr());
    };
    if (c.dim == 64) return bf16 ? go(kv4_attention_kernel<true, 64>) : go(kv4_attention_kernel<false, 64>);
    if (c.dim == 128) return bf16 ? go(kv4_attention_kernel<true, 128>) : go(kv4_attention_kernel<false, 128>);
    return bf16 ? go(kv4_attention_kernel<true, 256>) : go(kv4_attention_kernel<false, 256>);
}

}  // namespace bitnet
