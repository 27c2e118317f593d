// kv4_chunk.cu -- softmax attention over the 4-bit paged KV cache for many rows where kv4_prefill.cu has
// no kernel: fp32 calls, whose operands need 22 bits, and dim 256, whose outputs fill the tensor memory.
//
// Method: bitnet_v2_engine.py page, BitNetV2Attention.forward on the fake-quantised keys and
// values, as in kv4_attention.cu.
//
// A CTA takes 128 rows (new tokens x query heads) that share a key head, 16 to a warp, and walks
// their positions 64 at a time.  The codes of the next 64 are on their way while these are worked on; all warps
// turn them into fp16 tiles in shared memory, which every warp then multiplies its rows with
// (mma.sync, S and O in registers).  So a code is unpacked once for 128 rows; kv4_rows_kernel does it for 16.
//
// Chunks of 16 bytes stand in shared memory at their place ^ (row % 8), so that eight rows of one column meet no bank
// twice.  Each group of 8 dimensions stands in the order 0 4 1 5 2 6 3 7, as the nibbles come out of a
// word; queries are stored in the same order and outputs are put back.
//
// What bounds it: a prompt of 2048 tokens, 32 query heads on 8, takes 247 us in fp32 at dim 128 (two products to
// each of the formula's: 278 TFLOP/s of them) and 316 in bf16 at dim 256 (217 TFLOP/s), against 550 and 943 of
// kv4_rows_kernel.  The tensor cores' mma.sync path is busy for 50 and 39 % of the time; unpacking
// and the two barriers of a step are not covered by products, as one CTA fills an SM's registers.  Tried, and no
// faster: two steps' tiles with one barrier a step (1 and 5 % slower), products in groups of four sums.
#include "kv4.cuh"

#include <cuda_fp16.h>
#include <math_constants.h>

namespace bitnet {

namespace {

constexpr int kRows = 128, kPos = 64, kThreads = 256;
constexpr uint32_t kNowhere = 0xffffffffu;
// as in kv4_attention.cu
template <bool BF16>
constexpr float kOff = BF16 ? 6.0f : 13.0f;
template <bool BF16>
constexpr float kLag = BF16 ? 8.0f : 1.0f;
constexpr float kNone = -3.0e38f;
constexpr int kSplits = 8;  // parts of an item at most
constexpr float kKeyUnit = 0x1p-16f;  // as in kv4_prefill.cu
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct ChunkParams {
    const void *q;
    int64_t qts, qhs;
    int q_heads, group;
    int64_t T;
    Kv4Cache c;
    Kv4Batch bt;
    float scale;
    int causal, window;  // INT32_MAX: none
    int rows_min;        // sequences with fewer rows are another kernel's
    void *out;
    float *lse;
    int *status;
    int splits;      // CTAs that share an item's positions
    float *part;     // [items][splits][D + 2][128]: outputs, reference, sum
    int64_t *place;  // [items][128]: the rows' places in the output, -1 for none
    uint32_t magic[2];  // {0x64086408, 0x64806480}, as data: a logic instruction takes one constant
};

template <int D, bool BF16>
struct Smem {
    static constexpr int NP = BF16 ? 1 : 2;
    static constexpr uint32_t kRow = D * 2;  // bytes of a row of halves
    static constexpr uint32_t kQ = 0, kQPart = kRows * kRow;
    static constexpr uint32_t kK = kQ + NP * kQPart, kV = kK + kPos * kRow;
    static constexpr uint32_t kCodes = kV + kPos * kRow;           // keys, then values
    static constexpr uint32_t kSteps = kCodes + 2 * kPos * D / 2;  // key steps, value steps
    static constexpr uint32_t kPlaces = kSteps + 2 * kPos * 4;     // [2][64] rows of the cache
    static constexpr uint32_t kMeta = kPlaces + 2 * kPos * 4;      // two words of live positions, two maxima
    static constexpr uint32_t kBytes = kMeta + 16;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool TRANS>
__device__ __forceinline__ void load_tiles(uint32_t (&r)[4], uint32_t at) {  // four 8 x 8 tiles, a row's address from each lane
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(at)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(at)
                     : "memory");
}
__device__ __forceinline__ uint32_t h2(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return h2(__floats2half2_rn(lo, hi)); }
__device__ __forceinline__ uint32_t rest2(float lo, float hi, uint32_t rounded) {  // what pack2 left
    const float2 f = __half22float2(as_h2(rounded));
    return pack2(lo - f.x, hi - f.y);
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool on) {  // 16 bytes; zeros where !on
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// Tiles of rows of a sequence that this kernel takes.
__device__ __forceinline__ int tiles_of(const ChunkParams &p, int b) {
    const int a = max(0, __ldg(p.bt.starts + b));
    const int64_t n = min((int64_t)max(0, __ldg(p.bt.starts + b + 1) - a), max((int64_t)0, p.T - a));
    const int64_t rows = n * p.group;
    return rows < p.rows_min ? 0 : (int)((rows + kRows - 1) / kRows);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) kv4_chunk_kernel(const __grid_constant__ ChunkParams p) {
    using S = Smem<D, BF16>;
    constexpr int NP = S::NP;
    extern __shared__ __align__(128) char smem[];
    __shared__ int item_of[3];
    __shared__ int64_t scan[kThreads / 32];

    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t base = smem_u32(smem);

    // this CTA's rows: the item-th tile from the end over all sequences, tiles and heads, as later rows see more
    const int B = p.bt.batch;
    const int per = (B + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) mine += tiles_of(p, b);
    int64_t before = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, before, x);
        if (lane >= x) before += y;
    }
    if (lane == 31) scan[warp] = before;
    __syncthreads();
    int64_t total = 0;
    before -= mine;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? scan[w] : 0;
        total += scan[w];
    }
    const int item = blockIdx.x / p.splits, part = blockIdx.x - item * p.splits;
    const int64_t index = total * p.c.heads - 1 - item;
    if (index < 0) {  // the same for the whole CTA: the grid is made for the most items that T rows can be
        if (p.splits > 1 && part == 0 && tid < kRows) p.place[(int64_t)item * kRows + tid] = -1;
        return;
    }
    {
        const int64_t at = index / p.c.heads;
        if (at >= before && at < before + mine) {
            int64_t off = at - before;
            int b = tid * per;
            while (off >= tiles_of(p, b)) off -= tiles_of(p, b++);
            item_of[0] = b;
            item_of[1] = (int)off;
            item_of[2] = (int)(index % p.c.heads);
        }
    }
    __syncthreads();
    const int b = item_of[0], kh = item_of[2];
    const int first = max(0, __ldg(p.bt.starts + b));
    const int n = max(0, __ldg(p.bt.starts + b + 1) - first);
    const int len = max(0, __ldg(p.bt.lens + b));
    const int pos0 = len - n;  // of the sequence's first row
    const int cap = (int)min((int64_t)len, (int64_t)p.bt.max_pages << p.c.page_log2);
    const int rows = (int)(min((int64_t)n, p.T - first) * p.group);
    const int row0 = item_of[1] * kRows;
    const int row_last = min(row0 + kRows, rows) - 1;
    const int end = p.causal ? min(cap, pos0 + row_last / p.group + 1) : cap;
    const int begin = p.causal ? (int)max((int64_t)0, (int64_t)pos0 + row0 / p.group - p.window + 1) : 0;
    const int all_steps = max(0, (end - begin / kPos * kPos + kPos - 1) / kPos);
    const int from = (int)((int64_t)all_steps * part / p.splits);
    const int step0 = begin / kPos + from;
    const int steps = (int)((int64_t)all_steps * (part + 1) / p.splits) - from;
    if (tid == 0 && cap < len) record_status(p.status, (int)BITNET_ERR_INVALID_ARG);

    // places of the positions: a thread to a position, a page number ahead
    const uint32_t mask = (1u << p.c.page_log2) - 1;
    auto wanted = [&](int j) {
        const int at = (step0 + j) * kPos + tid;
        return tid < kPos && j < steps && at < end && at >= begin;
    };
    auto page_of = [&](int j) {
        const int at = ((step0 + j) * kPos + tid) >> p.c.page_log2;
        return wanted(j) && at < p.bt.max_pages ? __ldg(p.bt.table + (int64_t)b * p.bt.table_stride + at) : -1;
    };
    uint32_t *const places = reinterpret_cast<uint32_t *>(smem + S::kPlaces);
    auto publish = [&](int j, int page) {
        uint32_t r = kNowhere;
        if (wanted(j)) {
            if ((unsigned)page < (unsigned)p.c.pages)
                r = (((uint32_t)page * p.c.heads + kh) << p.c.page_log2) + (((step0 + j) * kPos + tid) & mask);
            else
                record_status(p.status, (int)BITNET_ERR_INVALID_ARG);
        }
        if (tid < kPos) places[(j & 1) * kPos + tid] = r;
    };
    constexpr int kChunks = D / 32;  // 16-byte pieces of a row of codes
    float ks = 0.0f, vs = 0.0f;      // of this thread's position
    uint32_t own = kNowhere;
    auto fetch = [&](int j) {  // codes and steps of step j, whose places are published
        if (j < steps) {
#pragma unroll
            for (int i = 0; i < (kPos * kChunks + kThreads - 1) / kThreads; ++i) {
                const int x = tid + i * kThreads;
                if (x >= kPos * kChunks) break;  // at dim 64
                const uint32_t r = places[(j & 1) * kPos + x / kChunks];
                const uint64_t at = (uint64_t)(r != kNowhere ? r : 0) * (D / 2) + x % kChunks * 16;
                copy_async(base + S::kCodes + x * 16, p.c.k_codes + at, r != kNowhere);
                copy_async(base + S::kCodes + kPos * D / 2 + x * 16, p.c.v_codes + at, r != kNowhere);
            }
            if (tid < kPos) {
                own = places[(j & 1) * kPos + tid];
                ks = own != kNowhere ? __ldg(p.c.k_step + own) : 0.0f;
                vs = own != kNowhere ? __ldg(p.c.v_step + own) : 0.0f;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    publish(0, page_of(0));
    publish(1, page_of(1));
    int page = page_of(2);

    // The queries: scaled by a power of two into [2^14, 2^15), with the sign of the scale, as one or two fp16.  D / 8 lanes
    // share a row; a warp brings its own 16.
    float factor[2];  // of the rows g and g + 8: the scale with log2 e, over the power of two
    {
        constexpr int L = D / 8, kSets = 16 * L / 32;
        const int piece = lane % L;
        float mine_f = 0.0f;  // of row `lane` of the warp
#pragma unroll 1
        for (int i = 0; i < kSets; ++i) {
            const int rr = i * (32 / L) + lane / L, rw = row0 + warp * 16 + rr;
            const int tok = rw / p.group, head = kh * p.group + (rw - tok * p.group);
            const int64_t at = rw < rows ? (int64_t)(first + tok) * p.qts + (int64_t)head * p.qhs + 8 * piece : 0;
            float x[8];
            if constexpr (BF16) {
                const uint4 u = rw < rows ? __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at)) : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) x[2 * e] = __uint_as_float(w[e] << 16), x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            } else {
                const float4 *const src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + at);
                const float4 u = rw < rows ? __ldg(src) : make_float4(0, 0, 0, 0), v = rw < rows ? __ldg(src + 1) : make_float4(0, 0, 0, 0);
                x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
            }
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const uint32_t up_bits = min(max(0x86000000u - (top & 0x7f800000u), 0x07000000u), 0x7e800000u);
            // a row that is not finite is NaN everywhere, as infinite scores of one sign alone would hide every position
            const float up = top > 0 && top < 0x7f800000u ? __uint_as_float(up_bits) : 1.0f;
            const float sup = top < 0x7f800000u ? (p.scale < 0.0f ? -up : up) : CUDART_NAN_F;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= sup;
            const uint32_t to = base + S::kQ + (warp * 16 + rr) * S::kRow + ((piece ^ (rr & 7)) << 4);
            const uint32_t h[4] = {pack2(x[0], x[4]), pack2(x[1], x[5]), pack2(x[2], x[6]), pack2(x[3], x[7])};
            sts128(to, h[0], h[1], h[2], h[3]);
            if constexpr (!BF16)
                sts128(to + S::kQPart, rest2(x[0], x[4], h[0]), rest2(x[1], x[5], h[1]), rest2(x[2], x[6], h[2]), rest2(x[3], x[7], h[3]));
            // 1 / up, a power of two
            const float f = fmaxf(fabsf(p.scale) * (kLog2e / kKeyUnit) * __uint_as_float(0x7f000000u - __float_as_uint(up)), 1.0e-37f);
#pragma unroll
            for (int k = 0; k < 32 / L; ++k) {
                const float y = __shfl_sync(0xffffffffu, f, k * L);
                if (lane == i * (32 / L) + k) mine_f = y;
            }
        }
        factor[0] = __shfl_sync(0xffffffffu, mine_f, g);
        factor[1] = __shfl_sync(0xffffffffu, mine_f, g + 8);
    }
    // positions that the rows g, g + 8 see, and those that all rows of the warp see
    const int my_row = row0 + warp * 16 + g;
    int my_end[2], my_begin[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int r = min(my_row + 8 * c, rows - 1), tok = r / p.group;
        my_end[c] = p.causal ? min(cap, pos0 + tok + 1) : cap;
        my_begin[c] = p.causal ? (int)max((int64_t)0, (int64_t)pos0 + tok - p.window + 1) : 0;
    }
    const int warp_first = min(row0 + warp * 16, rows - 1) / p.group, warp_last = min(row0 + warp * 16 + 15, rows - 1) / p.group;
    const int all_end = p.causal ? min(cap, pos0 + warp_first + 1) : cap;
    const int all_begin = p.causal ? (int)max((int64_t)0, (int64_t)pos0 + warp_last - p.window + 1) : 0;

    float o[D / 8][4], ref[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    uint32_t vexp = 0x0d000000u;  // 2^-101: O is in units of this power of two, which no value step so far is twice as large as
    const uint32_t magic[2] = {p.magic[0], p.magic[1]};
    // of the low and the high nibbles of keys (in units of kKeyUnit) and of values
    const __half2 one[2] = {__float2half2_rn(kKeyUnit), __float2half2_rn(1.0f)};
    const __half2 off[2] = {__float2half2_rn(-1032.0f * kKeyUnit), __float2half2_rn(-1032.0f)};
    const __half2 sixteenth[2] = {__float2half2_rn(0.0625f * kKeyUnit), __float2half2_rn(0.0625f)};
    const __half2 off16[2] = {__float2half2_rn(-72.0f * kKeyUnit), __float2half2_rn(-72.0f)};
    float *const k_steps = reinterpret_cast<float *>(smem + S::kSteps), *const v_steps = k_steps + kPos;
    uint32_t *const meta = reinterpret_cast<uint32_t *>(smem + S::kMeta);
    // what a lane's part of a tile of 8 x 8 loads is at: rows lane % 8 (+ 8), pieces 0 or 1
    const uint32_t q_at = base + S::kQ + (warp * 16 + (lane & 15)) * S::kRow;
    const uint32_t k_at = base + S::kK + ((lane & 7) + (lane >> 4 & 1) * 8) * S::kRow;
    const uint32_t v_at = base + S::kV + (lane & 15) * S::kRow;
    const uint32_t q_piece = lane >> 4 & 1, k_piece = lane >> 3 & 1, v_piece = lane >> 4 & 1, turn = lane & 7;

    __syncthreads();  // places
    fetch(0);
    for (int j = 0; j < steps; ++j) {
        const int at0 = (step0 + j) * kPos;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the codes are there, and every warp is done with the tiles before
        // codes to fp16
#pragma unroll 4
        for (int i = 0; i < kPos * D / 8 / kThreads; ++i) {
            const int x = tid + i * kThreads, r = x / (D / 8), c = x % (D / 8);
            const uint32_t to = base + S::kK + r * S::kRow + ((c ^ (r & 7)) << 4);
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(smem + S::kCodes + side * (kPos * D / 2) + x * 4), v = w >> 8;
                sts128(to + side * (S::kV - S::kK), h2(__hfma2(as_h2((w & 0x000F000Fu) ^ magic[0]), one[side], off[side])),
                       h2(__hfma2(as_h2((w & 0x00F000F0u) ^ magic[1]), sixteenth[side], off16[side])),
                       h2(__hfma2(as_h2((v & 0x000F000Fu) ^ magic[0]), one[side], off[side])),
                       h2(__hfma2(as_h2((v & 0x00F000F0u) ^ magic[1]), sixteenth[side], off16[side])));
            }
        }
        if (at0 == 0) {  // position 0 is kept at 8 bits
            const uint32_t r = places[(j & 1) * kPos];
            __syncthreads();
            if (r != kNowhere && tid < 2 * (D / 8)) {
                const int side = tid / (D / 8), c = tid % (D / 8);
                const char4 *const c8 = reinterpret_cast<const char4 *>((side ? p.c.v_bos : p.c.k_bos) + (int64_t)(r >> p.c.page_log2) * D + 8 * c);
                const char4 a = c8[0], e = c8[1];
                const float u = side ? 1.0f : kKeyUnit;
                sts128(base + S::kK + side * (S::kV - S::kK) + (c << 4), pack2(a.x * u, e.x * u), pack2(a.y * u, e.y * u),
                       pack2(a.z * u, e.z * u), pack2(a.w * u, e.w * u));
            }
        }
        if (warp < kPos / 32) {
            const uint32_t bits = __float_as_uint(vs) & 0x7f800000u;
            // a step that is not finite: NaN for the rows that see it, and for no others (see kv4_rows_kernel)
            const bool live = own != kNowhere, bad = live && max(bits, __float_as_uint(ks) & 0x7f800000u) == 0x7f800000u;
            k_steps[tid] = bad ? CUDART_NAN_F : ks;
            v_steps[tid] = bad ? 0.0f : vs;
            const uint32_t live_bits = __ballot_sync(0xffffffffu, live);
            const uint32_t most = __reduce_max_sync(0xffffffffu, bad ? 0u : bits);
            if (lane == 0) meta[warp] = live_bits, meta[2 + warp] = most;
        }
        __syncthreads();
        fetch(j + 1);  // its places are there since the step before
        // Slot j % 2 was last read for step j, before the barrier.
        publish(j + 2, page);
        page = page_of(j + 3);

        // S = Q K^T
        float s[kPos / 8][4];
#pragma unroll
        for (int i = 0; i < kPos / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t a[NP][4];
#pragma unroll
            for (int part2 = 0; part2 < NP; ++part2) load_tiles<false>(a[part2], q_at + part2 * S::kQPart + (((2 * k + q_piece) ^ turn) << 4));
#pragma unroll
            for (int i = 0; i < kPos / 16; ++i) {
                uint32_t f[4];
                load_tiles<false>(f, k_at + i * 16 * S::kRow + (((2 * k + k_piece) ^ turn) << 4));
#pragma unroll
                for (int part2 = NP - 1; part2 >= 0; --part2) {
                    mma_f16(s[2 * i], a[part2], f[0], f[1]);
                    mma_f16(s[2 * i + 1], a[part2], f[2], f[3]);
                }
            }
        }
        const uint32_t live[2] = {meta[0], meta[1]};
        const uint32_t next_vexp = min(max(vexp, max(meta[2], meta[3])), 0x7e000000u);
        const bool edge = at0 < all_begin || at0 + kPos > all_end || (live[0] & live[1]) != 0xffffffffu;
#pragma unroll
        for (int i = 0; i < kPos / 8; ++i) {
            const float2 k2 = *reinterpret_cast<const float2 *>(k_steps + 8 * i + 2 * t);
            s[i][0] *= k2.x, s[i][1] *= k2.y, s[i][2] *= k2.x, s[i][3] *= k2.y;
        }
        if (edge) {
#pragma unroll
            for (int i = 0; i < kPos / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int x = 8 * i + 2 * t + (e & 1), at = at0 + x;
                    if (!(live[i / 4] >> (x & 31) & 1) || at < my_begin[e >> 1] || at >= my_end[e >> 1]) s[i][e] = -CUDART_INF_F;
                }
        }
        float tops[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int i = 0; i < kPos / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) tops[e >> 1] = fmaxf(tops[e >> 1], s[i][e]);
        const bool over = fmaf(tops[0], factor[0], -ref[0]) > kOff<BF16> + kLag<BF16> || fmaf(tops[1], factor[1], -ref[1]) > kOff<BF16> + kLag<BF16>;
        if (__any_sync(0xffffffffu, over) || next_vexp != vexp) {
            const float units = __uint_as_float(vexp) * __uint_as_float(0x7f000000u - next_vexp);
            vexp = next_vexp;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float most = tops[c];
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                const float next = fmaf(most, factor[c], -ref[c]) > kOff<BF16> + kLag<BF16> ? fmaf(most, factor[c], -kOff<BF16>) : ref[c];
                const float a = ex2(ref[c] - next);
                ref[c] = next;
                l[c] *= a;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) o[i][2 * c] *= a * units, o[i][2 * c + 1] *= a * units;
            }
        }
        // weights, times the values' steps over a power of two that none so far is twice as large as (fp32: none of this step), as
        // the left operand of O = O + P V
        const uint32_t own_vexp = BF16 ? vexp : min(max(0x0d000000u, max(meta[2], meta[3])), 0x7e000000u);
        const float inv_unit = __uint_as_float(0x7f000000u - own_vexp);
        uint32_t a[BF16 ? 1 : kPos / 16][NP][4];
#pragma unroll
        for (int i = 0; i < kPos / 16; ++i) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float(&z)[4] = s[2 * i + half];
                const float2 v2 = *reinterpret_cast<const float2 *>(v_steps + 16 * i + 8 * half + 2 * t);
                const float v[2] = {v2.x * inv_unit, v2.y * inv_unit};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[e] = ex2(fmaf(z[e], factor[e >> 1], -ref[e >> 1]));
                    l[e >> 1] += z[e];
                    z[e] *= v[e & 1];
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t(&to)[NP][4] = a[BF16 ? 0 : i];
                    to[0][2 * half + c] = pack2(z[2 * c], z[2 * c + 1]);
                    if constexpr (!BF16) to[NP - 1][2 * half + c] = rest2(z[2 * c], z[2 * c + 1], to[0][2 * half + c]);
                }
            }
            if constexpr (BF16) {
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    uint32_t f[4];
                    load_tiles<true>(f, v_at + i * 16 * S::kRow + (((2 * d + v_piece) ^ turn) << 4));
                    mma_f16(o[2 * d], a[0][0], f[0], f[1]);
                    mma_f16(o[2 * d + 1], a[0][0], f[2], f[3]);
                }
            }
        }
        if constexpr (!BF16) {
            // The tensor cores cut where they add, so their sums end with the step: kept over 12,000 positions of one sign they
            // were low by 144 * 2^-24 of the output, over 30,000 by 450, and are by 2 so (for 2 to 4 % of the time).  In bf16
            // calls, where it would be 8 to 10 %, O stays in the products' own registers: values of one sign over 30,000 positions
            // are low by 1240 * 2^-24, where half a step of the output is 32,768 to 65,536.
            const float to_o = __uint_as_float(own_vexp) * __uint_as_float(0x7f000000u - vexp);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                float acc[2][4] = {};
#pragma unroll
                for (int i = 0; i < kPos / 16; ++i) {
                    uint32_t f[4];
                    load_tiles<true>(f, v_at + i * 16 * S::kRow + (((2 * d + v_piece) ^ turn) << 4));
#pragma unroll
                    for (int part2 = NP - 1; part2 >= 0; --part2) {
                        mma_f16(acc[0], a[i][part2], f[0], f[1]);
                        mma_f16(acc[1], a[i][part2], f[2], f[3]);
                    }
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[2 * d + x][e] = fmaf(to_o, acc[x][e], o[2 * d + x][e]);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    // the outputs: this lane's columns 2 t and 2 t + 1 of a group are its dimensions t and t + 4
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        l[c] += __shfl_xor_sync(0xffffffffu, l[c], 1);
        l[c] += __shfl_xor_sync(0xffffffffu, l[c], 2);
        const int r = my_row + 8 * c, tok = r / p.group;
        const int64_t place = r < rows ? (int64_t)(first + tok) * p.q_heads + kh * p.group + (r - tok * p.group) : -1;
        const float unit = __uint_as_float(vexp);
        if (p.splits > 1) {
            const int rr = r - row0;
            float *const dst = p.part + ((int64_t)item * p.splits + part) * (D + 2) * kRows + rr;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                dst[(8 * i + t) * kRows] = o[i][2 * c] * (unit / kSumUnit);
                dst[(8 * i + t + 4) * kRows] = o[i][2 * c + 1] * (unit / kSumUnit);
            }
            if (t == 0) {
                dst[D * kRows] = ref[c];
                dst[(D + 1) * kRows] = l[c];
                if (part == 0) p.place[(int64_t)item * kRows + rr] = place;
            }
        } else if (place >= 0) {
            const float inv = l[c] == 0.0f ? 0.0f : unit / l[c];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const int64_t d = place * D + 8 * i + t;
                const float x = o[i][2 * c] * inv, y = o[i][2 * c + 1] * inv;
                if constexpr (BF16) {
                    static_cast<__nv_bfloat16 *>(p.out)[d] = __float2bfloat16_rn(x);
                    static_cast<__nv_bfloat16 *>(p.out)[d + 4] = __float2bfloat16_rn(y);
                } else {
                    static_cast<float *>(p.out)[d] = x;
                    static_cast<float *>(p.out)[d + 4] = y;
                }
            }
            if (p.lse && t == 0) p.lse[place] = l[c] == 0.0f ? -CUDART_INF_F : (ref[c] + log2f(l[c])) * kLn2;
        }
    }
}

// Joins the parts of 32 rows of an item, in the order of the positions.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) kv4_chunk_join_kernel(const __grid_constant__ ChunkParams p) {
    constexpr int64_t kPart = (D + 2) * kRows;
    __shared__ float out[32][D + 1];
    __shared__ int64_t places[32];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = blockIdx.x / (kRows / 32), row = blockIdx.x % (kRows / 32) * 32 + lane;
    int64_t place = p.place[(int64_t)item * kRows + row];
    if (place >= p.T * p.q_heads) place = -1;  // a workspace that calls share at the same time can hold anything
    if (__syncthreads_and(place < 0)) return;  // nobody's rows, whose parts may not be written
    const float *const src = p.part + (int64_t)item * p.splits * kPart + row;
    // everything of a row at a time: the references and sums, then eight parts of four dimensions
    float w[kSplits], l[kSplits], top = kNone, sum = 0.0f;
#pragma unroll
    for (int s = 0; s < kSplits; ++s) {
        w[s] = s < p.splits ? src[s * kPart + D * kRows] : kNone;
        l[s] = s < p.splits ? src[s * kPart + (D + 1) * kRows] : 0.0f;
    }
#pragma unroll
    for (int s = 0; s < kSplits; ++s) top = fmaxf(top, w[s]);
#pragma unroll
    for (int s = 0; s < kSplits; ++s) w[s] = ex2(w[s] - top), sum = fmaf(w[s], l[s], sum);
    const float inv = sum == 0.0f ? 0.0f : kSumUnit / sum;
    if (warp == 0) {
        places[lane] = place;
        if (p.lse && place >= 0) p.lse[place] = sum == 0.0f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2;
    }
#pragma unroll
    for (int d0 = 0; d0 < D / 8; d0 += 4) {
        float v[4][kSplits];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int s = 0; s < kSplits; ++s) v[e][s] = s < p.splits ? src[s * kPart + (8 * (d0 + e) + warp) * kRows] : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y = 0.0f;
#pragma unroll
            for (int s = 0; s < kSplits; ++s) y = fmaf(w[s], v[e][s], y);
            out[lane][8 * (d0 + e) + warp] = y * inv;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * D; i += 256) {
        const int r = i / D, d = i % D;
        if (places[r] < 0) continue;
        const float y = out[r][d];
        if constexpr (BF16) static_cast<__nv_bfloat16 *>(p.out)[places[r] * D + d] = __float2bfloat16_rn(y);
        else static_cast<float *>(p.out)[places[r] * D + d] = y;
    }
}

template <int D, bool BF16>
cudaError_t launch_chunks(const ChunkParams &p, int64_t items, cudaStream_t s) {
    constexpr int kBytes = Smem<D, BF16>::kBytes;
    static bool allowed[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !allowed[dev]) {
        e = cudaFuncSetAttribute((const void *)kv4_chunk_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) allowed[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * p.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kv4_chunk_kernel<D, BF16>, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    cfg.gridDim = dim3((unsigned)(items * (kRows / 32)));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv4_chunk_join_kernel<D, BF16>, p);
}

// The most items (tiles of rows and key heads) that T rows can make: at most one tile of a sequence is not full.
int64_t most_items(int64_t T, int group, int heads, int batch, int rows_min) {
    const int64_t rows = T * group;
    return (rows / kRows + (rows / rows_min < batch ? rows / rows_min : (int64_t)batch)) * heads;
}
// Parts of split items: up to three of them to an SM.
int64_t most_splits(int64_t items) {
    const int64_t s = items > 0 ? (int64_t)3 * sm_count() / items : 0;
    return s < 1 ? 1 : (s > kSplits ? kSplits : s);
}

}  // namespace

size_t kv4_chunk_workspace(int64_t T, int group, int heads, int dim, int batch, int rows_min) {
    const int64_t items = most_items(T, group, heads, batch, rows_min), splits = most_splits(items);
    if (splits == 1) return 0;
    return (size_t)items * kRows * (splits * (dim + 2) * sizeof(float) + sizeof(int64_t));
}

cudaError_t launch_kv4_chunks(const void *q, bool bf16, int64_t T, int q_heads, int64_t qts, int64_t qhs, const Kv4Cache &c,
                              const Kv4Batch &bt, float scale, bool causal, int window, int rows_min, void *out, float *lse,
                              void *ws, cudaStream_t s) {
    ChunkParams p = {};
    p.q = q, p.qts = qts, p.qhs = qhs, p.q_heads = q_heads, p.group = q_heads / c.heads, p.T = T;
    p.c = c, p.bt = bt, p.scale = scale, p.causal = causal, p.window = window, p.rows_min = rows_min;
    p.out = out, p.lse = lse, p.status = device_status_ptr();
    p.magic[0] = 0x64086408u, p.magic[1] = 0x64806480u;
    const int64_t items = most_items(T, p.group, c.heads, bt.batch, rows_min);
    if (items == 0) return cudaSuccess;
    if (T * p.group > INT32_MAX - kRows || items * 8 > INT32_MAX) return cudaErrorInvalidConfiguration;
    // With few items the positions are split over several CTAs, as many as leave the SMs least idle; an item costs
    // as much as kCost steps to begin and to end, and a join as kJoin.  (700 tokens of one head: 47 us unsplit and 29 split in
    // fp32 at dim 128, 60 and 39 in bf16 at dim 256.)
    constexpr int kCost = 4, kJoin = 1;
    const int64_t steps = ceil_div((int64_t)bt.max_pages << c.page_log2, kPos), sms = sm_count();
    int64_t best = -1;
    p.splits = 1;
    for (int64_t n = 1; n <= most_splits(items) && (n == 1 || steps >= 2 * n); ++n) {
        const int64_t cost = ceil_div(items * n, sms) * (kCost + ceil_div(steps, n)) + (n > 1 ? kJoin : 0);
        if (best < 0 || cost < best) best = cost, p.splits = (int)n;
    }
    p.place = static_cast<int64_t *>(ws);
    p.part = reinterpret_cast<float *>(p.place + items * kRows);
    if (c.dim == 64) return bf16 ? cudaErrorInvalidValue : launch_chunks<64, false>(p, items, s);
    if (c.dim == 128) return bf16 ? cudaErrorInvalidValue : launch_chunks<128, false>(p, items, s);
    return bf16 ? launch_chunks<256, true>(p, items, s) : launch_chunks<256, false>(p, items, s);
}

}  // namespace bitnet
