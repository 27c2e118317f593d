// kv4.cu -- writing rows into the 4-bit paged KV cache and reading them back.
//
// Method: bitnet_v2_engine.py page, BitNetV2Attention._quantize_kv_head (Eq. 5/6), on rows
// of D values, two codes to a byte:
//   position 0:            code = RoundClip(127 x / (max|x| + eps), -128, 127), kept at 8 bits
//   positions >= 1, 4 bit: code = RoundClip(sqrt7 x / (mean|x| + eps), -8, 7)
//   positions >= 1, 3 bit: code = RoundClip(3 x / (max|x| + eps), -4, 3)
//   step = (stat + eps) / Q.
//
// Both kernels are HBM-bound: a row is read once and written once.  A lane owns 8
// neighbouring values (one 32-bit word of codes), so LPR = D / 8 lanes share a row and a
// warp takes 256 / D rows at a time; kIter such sets are loaded before the first is used.
// A CTA takes a few tokens and a part of their 2 * heads rows; it looks its tokens' places up
// once, into shared memory, while its first rows are on their way.
#include "kv4.cuh"

namespace bitnet {

namespace {

constexpr int kWarps = 8;
constexpr int kIter = 4;       // row sets in flight per warp
constexpr int kMaxTokens = 4;  // tokens of a CTA
template <int D>
constexpr int kPerCta = kWarps * (256 / D) * kIter;  // rows of a CTA

template <bool BF16>
__device__ __forceinline__ void load8(const void *x, int64_t i, float *v) {
    if constexpr (BF16) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(x) + i));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(x) + i);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// Where a token stands.
struct Place {
    int page;  // -1: nowhere
    int row;
    int pos;
};

__device__ __forceinline__ void locate_tokens(const Kv4Cache &c, const Kv4Batch &bt, int t0, int tokens, int64_t T,
                                              int *status, Place *place) {
    const int i = threadIdx.x;
    if (i < tokens) {
        Place p = {-1, 0, -1};
        int b, pos;
        if (t0 + i < T && kv4_locate(bt, t0 + i, b, pos)) {
            p.pos = pos;
            if (pos >= 0) {
                p.page = kv4_page(c, bt, b, pos, status);
                p.row = pos & ((1 << c.page_log2) - 1);
            }
        } else {
            p.pos = INT32_MIN;  // no sequence: outputs stay as they are
        }
        place[i] = p;
    }
    __syncthreads();
}

// A row of a CTA: its token (fastest, so that the rows of one warp lie side by side in the
// cache), head and side (0 keys, 1 values).
struct RowId {
    int tok, head, side;
    bool live;
};
__device__ __forceinline__ RowId row_id(int r, int tokens_log2, int heads, int rows) {
    RowId id;
    id.live = r < rows;
    id.tok = r & ((1 << tokens_log2) - 1);
    const int hs = r >> tokens_log2;
    id.side = hs >= heads;
    id.head = id.side ? hs - heads : hs;
    return id;
}

// A NaN in a row makes its step NaN, so that it is not lost.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it leaves rne(t) in the low mantissa bits

// Writing.  The code is decided in fp32 where that is safe and in fp64 otherwise: the fp32
// product t = x * (Q / scale) is within 16 roundings (7 adds in a lane, 5 in the tree, the
// mean's and scale's additions and divisions, the product) of the exact one, below 1e-6
// relative, so a t further than 1.25e-6 * max|code| from a half-integer rounds as the exact
// value does.  About 1 row in 200 of 4-bit rows has a value nearer than that, and its warp
// forms the statistic and the products again in fp64.
template <bool BF16, int D>
__global__ void __launch_bounds__(32 * kWarps)
kv4_write_kernel(const void *__restrict__ k, const void *__restrict__ v, int64_t T, int64_t kts, int64_t khs,
                 int64_t vts, int64_t vhs, Kv4Cache c, Kv4Batch bt, int bits, float eps, int tokens_log2, int rows,
                 int *status) {
    constexpr int LPR = D / 8, RP = 32 / LPR;
    __shared__ Place place[kMaxTokens];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = lane % LPR;
    const int t0 = blockIdx.x << tokens_log2;
    const int r0 = blockIdx.y * kPerCta<D> + warp * RP;
    float x[kIter][8];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const RowId id = row_id(r0 + it * kWarps * RP + lane / LPR, tokens_log2, c.heads, rows);
        if (id.live && t0 + id.tok < T) {
            load8<BF16>(id.side ? v : k, (t0 + id.tok) * (id.side ? vts : kts) + id.head * (id.side ? vhs : khs) + 8 * p,
                        x[it]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[it][e] = 0.0f;
        }
    }
    locate_tokens(c, bt, t0, 1 << tokens_log2, T, status, place);
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const int r = r0 + it * kWarps * RP;
        if (r >= rows) break;  // uniform in the warp
        const RowId id = row_id(r + lane / LPR, tokens_log2, c.heads, rows);
        const Place at = id.live ? place[id.tok] : Place{-1, 0, -1};
        // the rows of a warp may differ in kind; every lane takes the same shuffles
        const bool bos = at.pos == 0;
        const bool mean = !bos && bits == 4;
        float a = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) a = mean ? a + fabsf(x[it][e]) : max_nan(a, fabsf(x[it][e]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
            const float b = __shfl_xor_sync(0xffffffffu, a, o);
            a = mean ? a + b : max_nan(a, b);
        }
        const float q = bos ? 127.0f : (bits == 4 ? 2.64575131106459059f : 3.0f);
        const float lo = bos ? -128.0f : (bits == 4 ? -8.0f : -4.0f);
        const float scale = __fadd_rn(mean ? a * (1.0f / D) : a, eps);
        const float s = __fdiv_rn(q, scale);
        float step = __fdiv_rn(scale, q);
        float t[8];
        bool near = !(scale <= 3.0e38f && s <= 3.0e38f);  // beyond fp32
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y = s * x[it][e];
            const float z = fminf(fmaxf(y, lo), -1.0f - lo);
            t[e] = __fadd_rn(z, kMagic);
            near |= fabsf(fabsf(z - __fsub_rn(t[e], kMagic)) - 0.5f) < -1.25e-6f * lo;
        }
        const uint32_t nears = __ballot_sync(0xffffffffu, near);
        if (nears) {
            // only the rows that ask for it change, so that a row's step does not depend on its neighbours
            const bool mine = (nears >> (lane & ~(LPR - 1)) & (0xffffffffu >> (32 - LPR))) != 0;
            double w = 0.0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double m = fabs((double)x[it][e]);
                w = mean ? w + m : fmax(w, m);
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) {
                const double b = __shfl_xor_sync(0xffffffffu, w, o);
                w = mean ? w + b : fmax(w, b);
            }
            const double qd = bos ? 127.0 : (bits == 4 ? 2.6457513110645905905 : 3.0);
            const double sd = (mean ? w / D : w) + (double)eps;
            if (mine) step = scale != scale ? scale : (float)(sd / qd);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double y = fmin(fmax((double)x[it][e] * (qd / sd), (double)lo), -1.0 - (double)lo);
                if (mine) t[e] = __fadd_rn((float)rint(y), kMagic);
            }
        }
        if (at.page < 0) continue;
        const int64_t row = kv4_rows(c, at.page, id.head) + at.row;
        uint32_t w = 0, w0 = 0, w1 = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= (__float_as_uint(t[e]) & 15u) << (4 * e);
        *reinterpret_cast<uint32_t *>((id.side ? c.v_codes : c.k_codes) + row * (D / 2) + 4 * p) = w;
        if (p == 0) (id.side ? c.v_step : c.k_step)[row] = step;
        if (bos) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w0 |= (__float_as_uint(t[e]) & 255u) << (8 * e);
                w1 |= (__float_as_uint(t[e + 4]) & 255u) << (8 * e);
            }
            *reinterpret_cast<uint2 *>((id.side ? c.v_bos : c.k_bos) + ((int64_t)at.page * c.heads + id.head) * D + 8 * p) =
                make_uint2(w0, w1);
        }
    }
}

// Reading back: value = step * code.
template <bool BF16, int D>
__global__ void __launch_bounds__(32 * kWarps)
kv4_read_kernel(Kv4Cache c, Kv4Batch bt, int64_t T, void *__restrict__ k_out, void *__restrict__ v_out,
                int tokens_log2, int rows, int *status) {
    constexpr int LPR = D / 8, RP = 32 / LPR;
    __shared__ Place place[kMaxTokens];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = lane % LPR;
    const int t0 = blockIdx.x << tokens_log2;
    locate_tokens(c, bt, t0, 1 << tokens_log2, T, status, place);
    const int r0 = blockIdx.y * kPerCta<D> + warp * RP;
    uint32_t w[kIter];
    uint2 w8[kIter];
    float step[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const RowId id = row_id(r0 + it * kWarps * RP + lane / LPR, tokens_log2, c.heads, rows);
        const Place at = id.live ? place[id.tok] : Place{-1, 0, -1};
        w[it] = 0, step[it] = 0.0f, w8[it] = make_uint2(0, 0);
        if (at.page >= 0) {
            const int64_t row = kv4_rows(c, at.page, id.head) + at.row;
            step[it] = (id.side ? c.v_step : c.k_step)[row];
            if (at.pos == 0)
                w8[it] = *reinterpret_cast<const uint2 *>((id.side ? c.v_bos : c.k_bos) +
                                                          ((int64_t)at.page * c.heads + id.head) * D + 8 * p);
            else
                w[it] = *reinterpret_cast<const uint32_t *>((id.side ? c.v_codes : c.k_codes) + row * (D / 2) + 4 * p);
        }
    }
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const RowId id = row_id(r0 + it * kWarps * RP + lane / LPR, tokens_log2, c.heads, rows);
        if (!id.live) continue;
        const Place at = place[id.tok];
        void *out = id.side ? v_out : k_out;
        if (at.pos == INT32_MIN || !out) continue;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int code = at.pos == 0 ? (int)(int8_t)((e < 4 ? w8[it].x : w8[it].y) >> (8 * (e & 3)))
                                         : (int)(w[it] << (28 - 4 * e)) >> 28;
            y[e] = step[it] * (float)code;
        }
        const int64_t o = ((int64_t)(t0 + id.tok) * c.heads + id.head) * D + 8 * p;
        if constexpr (BF16) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
                h[e] = *reinterpret_cast<const uint32_t *>(&b);
            }
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(out) + o) = make_uint4(h[0], h[1], h[2], h[3]);
        } else {
            float4 *d = reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + o);
            d[0] = make_float4(y[0], y[1], y[2], y[3]);
            d[1] = make_float4(y[4], y[5], y[6], y[7]);
        }
    }
}

struct RowGrid {
    dim3 grid;
    int tokens_log2, rows;
};
// Tokens of a CTA: four where that leaves at least eight CTAs to an SM (neighbouring rows
// of the cache are then moved together), one otherwise.
RowGrid row_grid(int64_t T, int heads, int D) {
    RowGrid g;
    const int per_round = kWarps * (256 / D) * kIter;
    g.tokens_log2 = 0;
    while (g.tokens_log2 < 2 && ceil_div(T, 2 << g.tokens_log2) * ceil_div((int64_t)2 * heads << (g.tokens_log2 + 1), per_round) >=
                                    8 * (int64_t)sm_count())
        ++g.tokens_log2;
    g.rows = (2 * heads) << g.tokens_log2;
    g.grid = dim3((unsigned)ceil_div(T, 1 << g.tokens_log2), (unsigned)ceil_div(g.rows, per_round));
    return g;
}

template <typename... P, typename... A>
cudaError_t launch_rows(void (*kernel)(P...), dim3 grid, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_kv4_write(const void *k, const void *v, bool bf16, int64_t T, int64_t kts, int64_t khs, int64_t vts,
                             int64_t vhs, const Kv4Cache &c, const Kv4Batch &bt, int bits, float eps, cudaStream_t s) {
    const RowGrid g = row_grid(T, c.heads, c.dim);
    int *status = device_status_ptr();
    auto go = [&](auto kernel) {
        return launch_rows(kernel, g.grid, s, k, v, T, kts, khs, vts, vhs, c, bt, bits, eps, g.tokens_log2, g.rows,
                           status);
    };
    if (c.dim == 64) return bf16 ? go(kv4_write_kernel<true, 64>) : go(kv4_write_kernel<false, 64>);
    if (c.dim == 128) return bf16 ? go(kv4_write_kernel<true, 128>) : go(kv4_write_kernel<false, 128>);
    return bf16 ? go(kv4_write_kernel<true, 256>) : go(kv4_write_kernel<false, 256>);
}

cudaError_t launch_kv4_read(const Kv4Cache &c, const Kv4Batch &bt, int64_t T, void *k_out, void *v_out, bool bf16,
                            cudaStream_t s) {
    const RowGrid g = row_grid(T, c.heads, c.dim);
    int *status = device_status_ptr();
    auto go = [&](auto kernel) {
        return launch_rows(kernel, g.grid, s, c, bt, T, k_out, v_out, g.tokens_log2, g.rows, status);
    };
    if (c.dim == 64) return bf16 ? go(kv4_read_kernel<true, 64>) : go(kv4_read_kernel<false, 64>);
    if (c.dim == 128) return bf16 ? go(kv4_read_kernel<true, 128>) : go(kv4_read_kernel<false, 128>);
    return bf16 ? go(kv4_read_kernel<true, 256>) : go(kv4_read_kernel<false, 256>);
}

}  // namespace bitnet
