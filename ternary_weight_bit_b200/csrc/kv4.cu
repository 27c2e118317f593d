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
// warp takes 256 / D rows at a time; four such sets (reading: eight) are loaded before the first is used.
// A CTA takes a few tokens and a part of their heads, half of its warps the keys and half the
// values; it looks its tokens' places up once, into shared memory (a write's first rows are on
// their way meanwhile).
//
// Measured (bf16, dim 128): writing 14,157 rows of 32 key heads (277 MB) takes 84 us, 3.3 TB/s, bound by the
// issue of instructions (77 % of the slots, 150 to 8 values of a lane); reading 112,186 rows of 8 key heads back (524 MB)
// takes 99 us, 5.3 TB/s of a copy's 6.5.  Whole rows to a warp's registers in turns, with as many CTAs as fill the
// SMs once, was slower for reading (144 us, of registers) and no faster for writing.
#include <type_traits>

#include "kv4.cuh"

namespace bitnet {

namespace {

constexpr int kWarps = 8;
constexpr int kWriteIter = 4, kReadIter = 8;  // row sets in flight per warp
template <int D>
constexpr int kSet = kWarps / 2 * (256 / D);  // rows that a side's warps take at a time
template <int D>
constexpr int kMaxTokens = kSet<D> < 16 ? kSet<D> : 16;  // tokens of a CTA

// A lane's 8 values of a row, as they lie in memory.
template <bool BF16>
struct Raw {
    uint4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const char *x, bool on) {
        const uint4 *const p = reinterpret_cast<const uint4 *>(x);
#pragma unroll
        for (int j = 0; j < (BF16 ? 1 : 2); ++j) w[j] = on ? __ldg(p + j) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[BF16 ? 0 : 1].x, w[BF16 ? 0 : 1].y, w[BF16 ? 0 : 1].z, w[BF16 ? 0 : 1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = __uint_as_float(!BF16 ? u[j] : (j % 2 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16));
    }
};

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

// A lane's rows: those of one token and side, heads first, first + step, ...  The token goes
// fastest over the warps' rows, so that neighbouring rows of the cache are moved together.
// Where the heads are too FEW to fill a CTA so, it takes one head of kSet * ITER tokens: tok, tok + kSet, ...
template <int D, int ITER, bool FEW>
struct Rows {
    static constexpr int kTokens = FEW ? kSet<D> * ITER : kMaxTokens<D>;
    int tok, first, step;
    bool side;  // values
    __device__ __forceinline__ Rows(int tokens_log2) {
        const int warp = threadIdx.x >> 5;
        const int r = (warp & (kWarps / 2 - 1)) * (256 / D) + (threadIdx.x & 31) / (D / 8);
        if constexpr (FEW) {
            tok = r, first = blockIdx.y, step = 0;
        } else {
            const int of = blockIdx.y * (kSet<D> * ITER) + r;
            tok = of & ((1 << tokens_log2) - 1);
            first = of >> tokens_log2;
            step = kSet<D> >> tokens_log2;
        }
        side = __shfl_sync(0xffffffffu, warp, 0) >= kWarps / 2;
    }
    __device__ __forceinline__ int token(int it) const { return FEW ? tok + it * kSet<D> : tok; }
};

// A NaN in a row makes its step NaN, so that it is not lost.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it leaves rne(t) in the low mantissa bits

// Writing.  A code is decided in fp32 where that is safe and in fp64 otherwise.  In fp32 it is
// level = rne(n * u) with u = x / scale * (Q / n) + zero / n clamped to [0, 1] by the addition
// itself, n + 1 levels from -zero on.  u * n is off by at most 17 roundings of x Q / scale (7
// adds in a lane, 5 in the tree, the scale's addition, the reciprocal at two, the constant and
// its product), 17 * 2^-24 zero, and the roundings of u and zero / n, n 2^-24: together below
// 1.15e-6 zero.  So where n u is further than 1.25e-6 zero from a half-integer, its level is the
// exact value's.  (3 bits: a maximum has no roundings, which leaves 5, 0.42e-6 zero in all; halves of the
// maximum, frequent in bf16, are only 1.5 eps / max from a border.)  About 1 row in 200 of 4-bit rows has a value nearer than that; its warp, and
// that of a position 0, forms the statistic and the products again in fp64.
template <bool BF16, int D, int BITS, bool FEW>
__global__ void __launch_bounds__(32 * kWarps, BF16 ? 4 : 3)
kv4_write_kernel(const void *__restrict__ k, const void *__restrict__ v, int64_t T, int64_t kts, int64_t khs,
                 int64_t vts, int64_t vhs, Kv4Cache c, Kv4Batch bt, float eps, int tokens_log2, int *status) {
    constexpr int LPR = D / 8, kIter = kWriteIter;
    static_assert(kIter <= LPR, "lane i of a row keeps the step of iteration i");
    constexpr double kQ = BITS == 4 ? 2.6457513110645905905 : 3.0;
    constexpr float kZero = BITS == 4 ? 8.0f : 4.0f, kLevels = 2.0f * kZero - 1.0f, kNear = BITS == 4 ? 1.25e-6f : 0.45e-6f;
    using R = Rows<D, kIter, FEW>;
    __shared__ Place place[R::kTokens];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31;
    const int p = lane % LPR;
    const int t0 = FEW ? blockIdx.x * R::kTokens : blockIdx.x << tokens_log2;
    const R id(tokens_log2);
    const int heads = c.heads;
    int live = 0;  // the lane's heads; lane 0 has the warp's most
#pragma unroll
    for (int it = 0; it < kIter; ++it) live += id.first + it * id.step < heads;
    const int most_live = __shfl_sync(0xffffffffu, live, 0);
    Raw<BF16> raw[kIter];
    {
        constexpr int kSize = BF16 ? 2 : 4;
        const int64_t ts = id.side ? vts : kts, hs = id.side ? vhs : khs;
        const int count = FEW ? (int)min((int64_t)kIter, (T - t0 - id.tok + kSet<D> - 1) / kSet<D>) : (t0 + id.tok < T ? live : 0);
        const char *from = static_cast<const char *>(id.side ? v : k) + ((t0 + id.tok) * ts + id.first * hs + 8 * p) * kSize;
        const int64_t stride = (FEW ? kSet<D> * ts : id.step * hs) * kSize;
#pragma unroll
        for (int it = 0; it < kIter; ++it, from += stride) raw[it].load(from, it < count);
    }
    locate_tokens(c, bt, t0, FEW ? R::kTokens : 1 << tokens_log2, T, status, place);
    Place at = place[id.tok];
    int64_t first = kv4_rows(c, max(at.page, 0), id.first) + at.row;
    const int64_t stride = (int64_t)id.step << c.page_log2;
    uint8_t *const all_codes = id.side ? c.v_codes : c.k_codes;
    uint8_t *codes = all_codes + first * (D / 2) + 4 * p;
    float own = 0.0f;  // of iteration p: the scale, or the step where fp64 gave it
    bool is_step = false;
#pragma unroll
    for (int it = 0; it < kIter; ++it, codes += stride * (D / 2)) {
        if (it >= most_live) break;
        if (FEW && it > 0) {
            at = place[id.token(it)];
            first = kv4_rows(c, max(at.page, 0), id.first) + at.row;
            codes = all_codes + first * (D / 2) + 4 * p;
        }
        const int count = at.page >= 0 ? live : 0;
        const bool bos = at.pos == 0;
        float x[8], a = 0.0f;
        raw[it].values(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) a = BITS == 4 ? a + fabsf(x[e]) : max_nan(a, fabsf(x[e]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
            const float b = __shfl_xor_sync(0xffffffffu, a, o);
            a = BITS == 4 ? a + b : max_nan(a, b);
        }
        const float scale = __fadd_rn(BITS == 4 ? a * (1.0f / D) : a, eps);
        const float s = (float)(kQ / kLevels) * rcp(scale);
        float f[8], most = 0.0f;  // levels, and how far the farthest value is from its own
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = __saturatef(fmaf(x[e], s, kZero / kLevels));
            f[e] = __fsub_rn(fmaf(u, kLevels, kMagic), kMagic);
            most = fmaxf(most, fabsf(fmaf(u, kLevels, -f[e])));
        }
        // four levels to the low 16 bits of a float; level - zero in two's complement is (level + 8 - zero) ^ 8
        const float lo = fmaf(fmaf(fmaf(f[3] + 2048.0f, 16.0f, f[2]), 16.0f, f[1]), 16.0f, f[0]);
        const float hi = fmaf(fmaf(fmaf(f[7] + 2048.0f, 16.0f, f[6]), 16.0f, f[5]), 16.0f, f[4]);
        uint32_t w = (__byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410) + (BITS == 4 ? 0u : 0x44444444u)) ^ 0x88888888u;
        if (p == it) own = scale;
        const uint32_t asks = __ballot_sync(0xffffffffu, bos || !(scale >= 1e-36f && scale <= 1e36f && most < 0.5f - kNear * kZero));
        if (asks) {
            // the rows of a warp may differ in kind; every lane takes the same shuffles, and only
            // the rows that ask for it change, so that a row's step does not depend on its neighbours
            const bool mean = BITS == 4 && !bos;
            double sum = a;  // 3 bits: the maximum, exact already
            float nan = a;
            if constexpr (BITS == 4) {
                sum = 0.0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double m = fabs((double)x[e]);
                    sum = mean ? sum + m : fmax(sum, m);
                }
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) {
                    const double b = __shfl_xor_sync(0xffffffffu, sum, o);
                    sum = mean ? sum + b : fmax(sum, b);
                }
                nan = fabsf(x[0]);
#pragma unroll
                for (int e = 1; e < 8; ++e) nan = max_nan(nan, fabsf(x[e]));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) nan = max_nan(nan, __shfl_xor_sync(0xffffffffu, nan, o));
            }
            if (asks >> (lane & ~(LPR - 1)) & (0xffffffffu >> (32 - LPR))) {
                const double q = bos ? 127.0 : kQ, zero = bos ? 128.0 : (double)kZero;
                const double sd = (mean ? sum / D : sum) + (double)eps;
                if (p == it) own = nan != nan ? nan : (float)(sd / q), is_step = true;
                const double qs = q / sd;
                uint32_t w8[2] = {};
                w = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t code = (uint32_t)(int)rint(fmin(fmax((double)x[e] * qs, -zero), zero - 1.0));
                    w |= (code & 15u) << (4 * e);
                    w8[e >> 2] |= (code & 255u) << (8 * (e & 3));
                }
                if (bos && it < count)
                    *reinterpret_cast<uint2 *>((id.side ? c.v_bos : c.k_bos) + ((int64_t)at.page * heads + id.first + it * id.step) * D + 8 * p) =
                        make_uint2(w8[0], w8[1]);
            }
        }
        if (it < count) *reinterpret_cast<uint32_t *>(codes) = w;
    }
    if (FEW && p < kIter) {
        at = place[id.token(p)];
        first = kv4_rows(c, max(at.page, 0), id.first) + at.row;
    }
    if (p < live && at.page >= 0)
        (id.side ? c.v_step : c.k_step)[first + p * stride] = is_step ? own : __fdiv_rn(own, (float)kQ);
}

// Reading back: value = step * code.  Nibble e of a word plus 8, put into the mantissa of
// 2^(23 - 4 e), is that plus the nibble exactly; less 2^(23 - 4 e) + 8 it is the code.
// Lane p of a row writes values 8 p .. 8 p + 7 of it (bf16), or 4 p .. and 4 (p + D / 8) .. (fp32),
// so that a store's lanes lie side by side.
template <bool BF16, int D, bool FEW>
__global__ void __launch_bounds__(32 * kWarps)
kv4_read_kernel(Kv4Cache c, Kv4Batch bt, int64_t T, void *__restrict__ k_out, void *__restrict__ v_out,
                int tokens_log2, int *status) {
    constexpr int LPR = D / 8, kIter = kReadIter;
    using R = Rows<D, kIter, FEW>;
    __shared__ Place place[R::kTokens];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int p = (threadIdx.x & 31) % LPR;
    const int t0 = FEW ? blockIdx.x * R::kTokens : blockIdx.x << tokens_log2;
    const R id(tokens_log2);
    const int heads = c.heads;
    locate_tokens(c, bt, t0, FEW ? R::kTokens : 1 << tokens_log2, T, status, place);
    Place at = place[id.tok];
    void *const out = id.side ? v_out : k_out;
    if ((!FEW && at.pos == INT32_MIN) || !out) return;
    int64_t first = kv4_rows(c, max(at.page, 0), id.first) + at.row;
    const int64_t stride = (int64_t)id.step << c.page_log2;
    const uint8_t *const codes = id.side ? c.v_codes : c.k_codes;
    const float *const steps = id.side ? c.v_step : c.k_step;
    uint32_t w[kIter];
    float step[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        w[it] = 0u, step[it] = 0.0f;  // what is nowhere reads as 0 (of code 0: not -0)
        if (FEW && it > 0) {
            at = place[id.token(it)];
            first = kv4_rows(c, max(at.page, 0), id.first) + at.row;
        }
        if (at.page >= 0 && id.first + it * id.step < heads) {
            const int64_t row = FEW ? first : first + it * stride;
            const uint8_t *const from = codes + row * (D / 2);
            step[it] = steps[row];
            if constexpr (BF16) {
                w[it] = *reinterpret_cast<const uint32_t *>(from + 4 * p);
            } else {
                const uint16_t *const c16 = reinterpret_cast<const uint16_t *>(from) + p;
                w[it] = c16[0] | (uint32_t)c16[LPR] << 16;
            }
        }
    }
    const int64_t o = ((int64_t)(t0 + id.tok) * heads + id.first) * D + (BF16 ? 8 : 4) * p;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const int head = id.first + it * id.step;
        if (head >= heads) break;
        if (FEW) {
            at = place[id.token(it)];
            if (at.pos == INT32_MIN) continue;
        }
        const bool on = at.page >= 0, bos = at.pos == 0;
        const int64_t to = o + (FEW ? (int64_t)it * kSet<D> * heads * D : it * id.step * D);
        float y[8];
        if (bos) {
            const int8_t *const c8 = (id.side ? c.v_bos : c.k_bos) + ((int64_t)max(at.page, 0) * heads + head) * D;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = on ? step[it] * (float)c8[BF16 ? 8 * p + e : 4 * p + (e & 3) + (e >> 2) * (D / 2)] : 0.0f;
        } else {
            const uint32_t u[2] = {w[it] ^ 0x88888888u, (w[it] ^ 0x88888888u) >> 16};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t one = (uint32_t)(127 + 23 - 4 * (e & 3)) << 23;  // 2^(23 - 4 (e % 4)): its bit 4 (e % 4) counts 1
                const float base = __uint_as_float(one | 8u << (4 * (e & 3)));
                y[e] = step[it] * __fsub_rn(__uint_as_float((u[e >> 2] & (15u << (4 * (e & 3)))) | one), base);
            }
        }
        if constexpr (BF16) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
                h[e] = *reinterpret_cast<const uint32_t *>(&b);
            }
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(out) + to) = make_uint4(h[0], h[1], h[2], h[3]);
        } else {
            float *const d = reinterpret_cast<float *>(out) + to;
            *reinterpret_cast<float4 *>(d) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4 *>(d + D / 2) = make_float4(y[4], y[5], y[6], y[7]);
        }
    }
}

struct RowGrid {
    dim3 grid;
    int tokens_log2;
    bool few;
};
// Tokens of a CTA: as many as fill a CTA, and at least eight (neighbouring rows of the cache
// are then moved together), as long as that leaves eight CTAs to an SM.  Few heads that do not
// fill a CTA so have CTAs of their own, with more tokens (one head of 524,288 rows of dim 128 in bf16 is read at 5000 GB/s
// instead of 1900 and written at 3300 instead of 1650).
RowGrid row_grid(int64_t T, int heads, int D, int iter) {
    const int set = kWarps / 2 * (256 / D), per_cta = set * iter, most = set < 16 ? set : 16;
    auto fills = [](dim3 g) { return (int64_t)g.x * g.y >= 8 * (int64_t)sm_count(); };
    const dim3 few((unsigned)ceil_div(T, per_cta), (unsigned)heads);
    if (heads * most < per_cta && fills(few)) return {few, 0, true};
    auto grid = [&](int log2) { return dim3((unsigned)ceil_div(T, 1 << log2), (unsigned)ceil_div((int64_t)heads << log2, per_cta)); };
    int tokens_log2 = 0;
    for (int log2 = 1; (1 << log2) <= most && (log2 <= 3 || heads << log2 <= per_cta); ++log2)
        if (fills(grid(log2))) tokens_log2 = log2;
    return {grid(tokens_log2), tokens_log2, false};
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
    const RowGrid g = row_grid(T, c.heads, c.dim, kWriteIter);
    int *status = device_status_ptr();
    auto go = [&](auto kernel) { return launch_rows(kernel, g.grid, s, k, v, T, kts, khs, vts, vhs, c, bt, eps, g.tokens_log2, status); };
    auto of = [&](auto type, auto n, auto few) {
        constexpr bool kBf16 = decltype(type)::value, kFew = decltype(few)::value;
        constexpr int kBits = decltype(n)::value;
        if (c.dim == 64) return go(kv4_write_kernel<kBf16, 64, kBits, kFew>);
        if (c.dim == 128) return go(kv4_write_kernel<kBf16, 128, kBits, kFew>);
        return go(kv4_write_kernel<kBf16, 256, kBits, kFew>);
    };
    auto with = [&](auto type, auto n) { return g.few ? of(type, n, std::true_type()) : of(type, n, std::false_type()); };
    using std::integral_constant;
    if (bits == 4) return bf16 ? with(std::true_type(), integral_constant<int, 4>()) : with(std::false_type(), integral_constant<int, 4>());
    return bf16 ? with(std::true_type(), integral_constant<int, 3>()) : with(std::false_type(), integral_constant<int, 3>());
}

cudaError_t launch_kv4_read(const Kv4Cache &c, const Kv4Batch &bt, int64_t T, void *k_out, void *v_out, bool bf16,
                            cudaStream_t s) {
    const RowGrid g = row_grid(T, c.heads, c.dim, kReadIter);
    int *status = device_status_ptr();
    auto go = [&](auto kernel) {
        return launch_rows(kernel, g.grid, s, c, bt, T, k_out, v_out, g.tokens_log2, status);
    };
    auto of = [&](auto type, auto few) {
        constexpr bool kBf16 = decltype(type)::value, kFew = decltype(few)::value;
        if (c.dim == 64) return go(kv4_read_kernel<kBf16, 64, kFew>);
        if (c.dim == 128) return go(kv4_read_kernel<kBf16, 128, kFew>);
        return go(kv4_read_kernel<kBf16, 256, kFew>);
    };
    auto with = [&](auto type) { return g.few ? of(type, std::true_type()) : of(type, std::false_type()); };
    return bf16 ? with(std::true_type()) : with(std::false_type());
}

}  // namespace bitnet
