// kv4_prefill.cu -- softmax attention over the 4-bit paged KV cache for many rows (prompts and
// chunks of prompts), on the tcgen05 tensor cores.
//
// Method: bitnet_v2_engine.py page, BitNetV2Attention.forward on the fake-quantised keys and
// values, as in kv4_attention.cu: s_t = scale * kstep_t * (q . kcode_t),
// out = sum_t e^(s_t) vstep_t vcode_t / sum_t e^(s_t).
//
// A CTA takes 256 rows (new tokens x query heads) that share a key head, as two tiles of 128,
// and walks their positions 128 at a time:
//
//   warps 0-3, 4-7   softmax of tile 0, tile 1: a thread owns a row
//   warps 8-11       key codes -> fp16 in shared memory, a thread to a position; places and steps
//   warp 12          issues the products
//   warps 13-15      value codes -> fp16
//
//   S_w = Q_w K^T      both operands in shared memory, K-major, 128-byte swizzle; S in TMEM
//   P_w                fp16 weights, stored by the softmax warps over the first half of S_w
//   O_w += P_w V       P from TMEM, V in shared memory with the dimensions contiguous
//
// While one tile's softmax runs, the tensor cores work for the other.  The codes are exact in
// fp16; steps are fp32 factors of the scores' and the weights' columns.  Each group of 8 dimensions
// stands in shared memory in the order 0 4 1 5 2 6 3 7, as the nibbles come out of a word; queries
// are stored in the same order and outputs are put back.
//
// O stays in the tensor memory through all positions of an item's part.  The tensor cores cut where they add, so values of one
// sign come out low by about 3e-9 to a position: 1500 * 2^-24 over 30,000, where half a step of a bf16 output is 32,768 to
// 65,536.  (Sums that end with a step would move O through registers in each.)
//
// As in kv4_attention.cu, a row's reference moves only when a score passes it by more than kLag,
// and value steps are divided by a power of two that no step so far is twice as large as; O is
// rescaled in TMEM in those rare cases alone.
//
// What bounds it: a step (both tiles, 128 positions) takes 5700 cycles at dim 128 and 4400 at dim 64, of which
// the exponentials hold their unit for 2048 and the products the tensor cores for 1700; the rest is the chain
// product - load - maximum - exponentials - store - product of each tile, which the other tile's covers in part.  (S and
// O of two tiles fill the tensor memory at dim 128.  Within a tile, the product with V could begin before the last
// exponential, and S be loaded again instead of held in registers: not tried.)  Beginning and ending an item takes 6 to 10 us
// more.  Prompts of 4100, 1999 and 3298 tokens, 32 query heads on 8 of dim 128: 427 us, 608 TFLOP/s.  1024 and 637
// tokens at the ends of 16500 and 13719 at dim 64: 458 us, 446 TFLOP/s.  Tried, and no faster: S in two halves of 64
// positions in turns, 16 warps of softmax, exponentials by a polynomial on the fp32 units, weights in columns
// of their own at dim 64.
#include "kv4.cuh"

#include <cuda_fp16.h>
#include <math_constants.h>

#include <type_traits>

namespace bitnet {

namespace {

constexpr int kRows = 128;   // rows of a tile
constexpr int kPos = 128;    // positions of a step
constexpr int kThreads = 512;
constexpr int kValueThreads = 96;
constexpr int kKS = 2, kVS = 2, kStepStages = 4, kPlaceStages = 8;
// Registers of a thread of the two halves of the block, 256 threads each; what either lacks is spilled to an L1 that
// shared memory leaves little of (prompts at dim 128: 472 us with 192 and 64, 420 with 184 and 72, 453 with 176 and
// 80; a chunk at dim 64: 454, 518, 531).
template <int D>
constexpr int kSoftmaxRegs = D == 128 ? 184 : 192;
template <int D>
constexpr int kOtherRegs = 256 - kSoftmaxRegs<D>;
constexpr uint32_t kNowhere = 0xffffffffu;
constexpr float kOff = 6.0f, kLag = 8.0f, kNone = -3.0e38f;
constexpr int kSplits = 8;  // parts of an item at most
// Key codes stand in this unit (exactly: fp16 has multiples of 2^-24), which the rows' factors undo: products with queries of up to
// 2^15 stay below 2^14, so that with their key's step they pass fp32's range only where that is over 2^114.
constexpr float kKeyUnit = 0x1p-16f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// n / d for 0 <= n < 2^31 by a multiplication: with 2^l >= d, m = floor(2^32 (2^l - d) / d) + 1.
struct Divide {
    uint32_t mul, shift;
    __device__ __forceinline__ int operator()(int n) const { return (int)((__umulhi(mul, (uint32_t)n) + (uint32_t)n) >> shift); }
};
Divide divide_by(uint32_t d) {
    uint32_t l = 0;
    while ((1u << l) < d) ++l;
    return Divide{(uint32_t)((((uint64_t)1 << 32) * ((1ull << l) - d)) / d + 1), l};
}

struct TileParams {
    const void *q;
    int64_t qts, qhs;
    int q_heads, group;
    int64_t T;
    Kv4Cache c;
    Kv4Batch bt;
    float scale;
    int causal, window;  // INT32_MAX: none
    int rows_min;        // sequences with fewer rows are another kernel's
    uint16_t *out;
    float *lse;
    int *status;
    int splits;     // CTAs that share an item's positions
    float *part;    // [items][splits][D + 2][256]: outputs, reference, sum
    int64_t *place;  // [items][256]: the rows' places in the output, -1 for none
    Divide by_group;
    uint32_t magic[2];  // {0x64086408, 0x64806480}, as data: a logic instruction takes one constant
};

// Whether the two tiles take turns at the exponentials, so that one is at them while the other has its products
// and its maxima.  At dim 64 the products are short and both tiles fall into step without it (a chunk of 1661
// rows over 28000 positions: 591 us without turns, 522 with); at dim 128 the products keep them apart (440 and 460 us
// for prompts of 9397 rows).
template <int D>
constexpr bool kTurns = D == 64;

template <int D>
struct Smem {
    static constexpr int kTile = kRows * D * 2;  // bytes of a tile of Q, K or V
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kKS * kTile;
    static constexpr int kSteps = kV + kVS * kTile;            // [kStepStages][2][128] floats: key steps, value ratios
    static constexpr int kMeta = kSteps + kStepStages * 1024;  // [kStepStages][8]: 4 words of live positions, the power of two
    static constexpr int kPlaces = kMeta + kStepStages * 32;   // [kPlaceStages][128]: the positions' rows in the cache
    static constexpr int kFactors = kPlaces + kPlaceStages * 512;  // [256]: the rows' factors of their scores
    static constexpr int kOuts = kFactors + 2 * kRows * 4;         // [256] int64: the rows' places in the output, -1 for none
    static constexpr int kBars = kOuts + 2 * kRows * 8;
    static constexpr int kNumBars = 2 * kKS + 2 * kVS + kStepStages + kPlaceStages + 2 + 2 + 2 + 2;
    static constexpr int kSlot = kBars + 8 * kNumBars;
    static constexpr int kUsed = kSlot + 16 + 1024;  // and alignment
    static constexpr int kBytes = D == 128 ? 231424 : 160 * 1024;
    static_assert(kUsed <= kBytes && kBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two floats in one register pair.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(f2 x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// x = -inf where !seen.  Volatile, so that it stays inside its branch: as selects the masks of all steps
// were formed, 4 instructions to a score.
__device__ __forceinline__ void hide_unless(float &x, uint32_t seen) {
    asm volatile("{.reg .pred p; setp.ne.u32 p, %1, 0; selp.f32 %0, %0, 0fFF800000, p;}" : "+f"(x) : "r"(seen));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t h2(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A 128-byte-swizzled tile of rows of 64 halves.  K-major (Q, K): a row is 64 of the summed
// dimension, the next 8 rows lie 1024 bytes on.  Dimensions contiguous (V): a row is one position, the next 8
// positions lie 1024 bytes on, the next 64 dimensions kRows rows on.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, bool mn) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(mn ? (kRows * 128) >> 4 : 1) << 16;  // leading byte offset: the next 64 dimensions (V); unused (Q, K)
    d |= (uint64_t)(1024 >> 4) << 32;           // stride byte offset: the next 8 rows
    d |= (uint64_t)1 << 46;                     // descriptor version (sm100)
    d |= (uint64_t)2 << 61;                     // swizzle: 128B
    return d;
}
// D = f32, A = B = f16, M = 128.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
// Called by a converged warp; one lane issues.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
}

// Eight codes of a word as 16 bytes of fp16, dimensions in the order 0 4 1 5 2 6 3 7 (see halves() in
// kv4_attention.cu), times kKeyUnit for keys.
template <bool KEYS>
__device__ __forceinline__ void put_codes(uint32_t dst, uint32_t w, const uint32_t (&magic)[2]) {
    constexpr float kUnit = KEYS ? kKeyUnit : 1.0f;
    const uint32_t v = w >> 8;
    const __half2 one = __float2half2_rn(kUnit), off = __float2half2_rn(-1032.0f * kUnit);
    const __half2 sixteenth = __float2half2_rn(0.0625f * kUnit), off16 = __float2half2_rn(-72.0f * kUnit);
    auto low = [&](uint32_t x) { return KEYS ? __hfma2(as_h2(x), one, off) : __hadd2(as_h2(x), off); };
    sts128(dst, h2(low((w & 0x000F000Fu) ^ magic[0])), h2(__hfma2(as_h2((w & 0x00F000F0u) ^ magic[1]), sixteenth, off16)),
           h2(low((v & 0x000F000Fu) ^ magic[0])), h2(__hfma2(as_h2((v & 0x00F000F0u) ^ magic[1]), sixteenth, off16)));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_tiles_kernel(const __grid_constant__ TileParams p) {
    using S = Smem<D>;
    extern __shared__ char smem_raw[];
    __shared__ int item_of[4];
    __shared__ int64_t scan[kThreads / 32];

    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    char *const smem_base = smem_raw + (base - smem_u32(smem_raw));

    // this CTA's 256 rows: the blockIdx-th from the end over all sequences, pairs of tiles and heads
    const int B = p.bt.batch;
    const int per = (B + kThreads - 1) / kThreads;
    auto pairs_of = [&](int b) {
        const int a = max(0, __ldg(p.bt.starts + b));
        const int64_t n = min((int64_t)max(0, __ldg(p.bt.starts + b + 1) - a), max((int64_t)0, p.T - a));
        const int64_t rows = n * p.group;
        return rows < p.rows_min ? 0 : (int)((rows + 2 * kRows - 1) / (2 * kRows));
    };
    int64_t mine = 0;
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) mine += pairs_of(b);
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
        if (p.splits > 1 && part == 0 && tid < 2 * kRows) p.place[(int64_t)item * (2 * kRows) + tid] = -1;
        return;
    }
    {
        const int64_t at = index / p.c.heads;
        if (at >= before && at < before + mine) {
            int64_t off = at - before;
            int b = tid * per;
            while (off >= pairs_of(b)) off -= pairs_of(b++);
            item_of[0] = b;
            item_of[1] = (int)off;
            item_of[2] = (int)(index % p.c.heads);
        }
    }
    const uint32_t bars = base + S::kBars;
    const uint32_t k_full = bars, k_empty = k_full + 8 * kKS, v_full = k_empty + 8 * kKS, v_empty = v_full + 8 * kVS,
                   st_full = v_empty + 8 * kVS, s_full = st_full + 8 * kStepStages, p_full = s_full + 16, turn = p_full + 16, q_full = turn + 16,
                   o_full = q_full + 8, at_full = o_full + 8;
    if (tid == 0) {
        auto init = [&](uint32_t bar, int n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(n) : "memory");
        };
        for (int i = 0; i < kKS; ++i) init(k_full + 8 * i, 128), init(k_empty + 8 * i, 1);
        for (int i = 0; i < kVS; ++i) init(v_full + 8 * i, kValueThreads), init(v_empty + 8 * i, 1);
        for (int i = 0; i < kStepStages; ++i) init(st_full + 8 * i, 128);
        for (int i = 0; i < kPlaceStages; ++i) init(at_full + 8 * i, 128);
        for (int w = 0; w < 2; ++w) init(s_full + 8 * w, 1), init(p_full + 8 * w, 128), init(turn + 8 * w, 128);
        init(q_full, 256);
        init(o_full, 1);
        fence_mbar_init();
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + S::kSlot), "r"(512) : "memory");
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lds32(base + S::kSlot);
    const int b = item_of[0], kh = item_of[2];

    const int first = max(0, __ldg(p.bt.starts + b));
    const int n = max(0, __ldg(p.bt.starts + b + 1) - first);
    const int len = max(0, __ldg(p.bt.lens + b));
    const int pos0 = len - n;  // of the sequence's first row
    const int cap = (int)min((int64_t)len, (int64_t)p.bt.max_pages << p.c.page_log2);
    const int rows = (int)(min((int64_t)n, p.T - first) * p.group);
    const int row0 = item_of[1] * 2 * kRows;
    const int row_last = min(row0 + 2 * kRows, rows) - 1;
    const int end = p.causal ? min(cap, pos0 + row_last / p.group + 1) : cap;
    const int begin = p.causal ? (int)max((int64_t)0, (int64_t)pos0 + row0 / p.group - p.window + 1) : 0;
    const int all_steps = max(0, (end - begin / kPos * kPos + kPos - 1) / kPos);
    const int from = (int)((int64_t)all_steps * part / p.splits);
    const int step0 = begin / kPos + from;
    const int steps = (int)((int64_t)all_steps * (part + 1) / p.splits) - from;
    if (tid == 0 && cap < len) record_status(p.status, (int)BITNET_ERR_INVALID_ARG);

    if (warp < 8) {
        // ---------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs<D>));
        const int w = warp >> 2;
        const int r = tid & 127;                     // row of the tile, and lane of TMEM
        const int row = row0 + w * kRows + r;        // row of the sequence
        const bool on = row < rows;
        const int tok = p.by_group(row);
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_off + w * kPos, t_o = tmem + lane_off + 2 * kPos + w * D;

        // The tile's queries: scaled by a power of two into [2^14, 2^15), with the sign of the scale, in fp16.  D / 8 lanes
        // share a row.
        {
            constexpr int L = D / 8, kSets = kRows * L / 128;
            const int piece = lane % L;
            const uint32_t mine = base + S::kQ + w * S::kTile + (piece >> 3) * (kRows * 128);
            auto row_at = [&](int i) { return (i * 4 + (warp & 3)) * (32 / L) + lane / L; };
            auto at = [&](int rr) { return mine + rr * 128 + (((piece & 7) ^ (rr & 7)) << 4); };
            // each lane brings its 8 values to where their fp16 belongs, ...
#pragma unroll 4
            for (int i = 0; i < kSets; ++i) {
                const int rr = row_at(i), rw = row0 + w * kRows + rr;
                const int tk = p.by_group(rw), head = kh * p.group + (rw - tk * p.group);
                const uint16_t *const src = reinterpret_cast<const uint16_t *>(p.q) +
                                            (rw < rows ? (int64_t)(first + tk) * p.qts + (int64_t)head * p.qhs + 8 * piece : 0);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(rr)), "l"(src), "r"(rw < rows ? 16 : 0) : "memory");
                if (piece == 0)
                    *reinterpret_cast<int64_t *>(smem_base + S::kOuts + 8 * (w * kRows + rr)) =
                        rw < rows ? (int64_t)(first + tk) * p.q_heads + head : -1;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            // ... and turns them into it there
#pragma unroll 4
            for (int i = 0; i < kSets; ++i) {
                const int rr = row_at(i);
                uint32_t x[4], top = 0;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at(rr)) : "memory");
#pragma unroll
                for (int j = 0; j < 4; ++j) top = max(top, max((x[j] << 16) & 0x7fffffffu, x[j] & 0x7fff0000u));
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const uint32_t up_bits = min(max(0x86000000u - (top & 0x7f800000u), 0x07000000u), 0x7e800000u);
                // a row that is not finite is NaN everywhere, as infinite scores of one sign alone would hide every position
                const float up = top > 0 && top < 0x7f800000u ? __uint_as_float(up_bits) : 1.0f;
                const float sup = top < 0x7f800000u ? (p.scale < 0.0f ? -up : up) : CUDART_NAN_F;
                float y[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[2 * j] = __uint_as_float(x[j] << 16) * sup;
                    y[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u) * sup;
                }
                sts128(at(rr), pack2(y[0], y[4]), pack2(y[1], y[5]), pack2(y[2], y[6]), pack2(y[3], y[7]));
                if (piece == 0)  // 1 / up, a power of two
                    sts32(base + S::kFactors + 4 * (w * kRows + rr),
                          __float_as_uint(fmaxf(fabsf(p.scale) * (kLog2e / kKeyUnit) * __uint_as_float(0x7f000000u - __float_as_uint(up)), 1.0e-37f)));
            }
            fence_proxy_async_smem();
            arrive(q_full);
        }
        bool ok = mbar_wait_warp(q_full, 0, p.status);
        const float f = __uint_as_float(lds32(base + S::kFactors + 4 * (w * kRows + r)));  // of this row's scores, with log2 e

        // positions that this row sees, and those that all rows of the tile see
        const int tile_first = p.by_group(row0 + w * kRows), tile_last = min(row0 + (w + 1) * kRows, rows) - 1;
        const int my_end = p.causal && on ? pos0 + tok + 1 : INT32_MAX;
        const int my_begin = p.causal && on ? (int)max((int64_t)0, (int64_t)pos0 + tok - p.window + 1) : 0;
        const int all_end = p.causal ? min(cap, pos0 + tile_first + 1) : cap;
        const int all_begin = p.causal ? (int)max((int64_t)0, (int64_t)pos0 + tile_last / p.group - p.window + 1) : 0;

        float ref = kNone;
        f2 l2[4] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f), pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
        uint32_t vexp = 0x3f800000u;
        for (int j = 0; j < steps && ok; ++j) {
            const int at0 = (step0 + j) * kPos;
            const int st = j % kStepStages;
            if (!mbar_wait_warp(s_full + 8 * w, j & 1, p.status) || !mbar_wait_warp(st_full + 8 * st, (j / kStepStages) & 1, p.status)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t meta = base + S::kMeta + st * 32;
            const float4 *const k4 = reinterpret_cast<const float4 *>(smem_base + S::kSteps + st * 1024), *const v4 = k4 + 32;
            float s[kPos];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(t_s + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
            const uint32_t live[4] = {lds32(meta), lds32(meta + 4), lds32(meta + 8), lds32(meta + 12)};
            const uint32_t vexp_new = lds32(meta + 16);
            tmem_wait_ld();
            f2 z[kPos / 2];
#pragma unroll
            for (int i = 0; i < kPos / 4; ++i) {
                const float4 k = k4[i];
                z[2 * i] = mul2(pair(s[4 * i], s[4 * i + 1]), pair(k.x, k.y));
                z[2 * i + 1] = mul2(pair(s[4 * i + 2], s[4 * i + 3]), pair(k.z, k.w));
            }
            const bool edge = at0 < all_begin || at0 + kPos > all_end || (live[0] & live[1] & live[2] & live[3]) != 0xffffffffu;
            if (edge) {
                const int lo = my_begin - at0, hi = my_end - at0;  // bits lo .. hi - 1
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int a = min(max(lo - 32 * c, 0), 32), e = min(max(hi - 32 * c, 0), 32);
                    uint32_t m = live[c];
                    m &= e >= 32 ? 0xffffffffu : (1u << e) - 1u;
                    m &= a >= 32 ? 0u : ~((1u << a) - 1u);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x, y;
                        split(z[16 * c + i], x, y);
                        hide_unless(x, m & (1u << (2 * i)));
                        hide_unless(y, m & (2u << (2 * i)));
                        z[16 * c + i] = pair(x, y);
                    }
                }
            }
            float tops[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int i = 0; i < kPos / 2; ++i) {
                float x, y;
                split(z[i], x, y);
                tops[i & 3] = fmaxf(tops[i & 3], fmaxf(x, y));
            }
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            const bool over = fmaf(top, f, -ref) > kOff + kLag;
            bool rescale = false;
            float factor = 1.0f;
            if (__any_sync(0xffffffffu, over) || vexp_new != vexp) {
                const float next = over ? fmaf(top, f, -kOff) : ref;
                const float a = ex2(ref - next);
                ref = next;
#pragma unroll
                for (int i = 0; i < 4; ++i) l2[i] = mul2(l2[i], pair(a, a));
                // vexp / vexp_new, both powers of two
                rescale = j > 0;
                factor = a * __uint_as_float(vexp) * __uint_as_float(0x7f000000u - vexp_new);
                vexp = vexp_new;
            }
            if (kTurns<D> && (w == 1 || j > 0) && !mbar_wait_warp(turn + 8 * w, (w == 1 ? j : j - 1) & 1, p.status)) {
                ok = false;
                break;
            }
            const f2 ff = pair(f, f), nref = pair(-ref, -ref);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t h[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 v = v4[8 * c + i];
                    float x[4];
                    split(fma2(z[16 * c + 2 * i], ff, nref), x[0], x[1]);
                    split(fma2(z[16 * c + 2 * i + 1], ff, nref), x[2], x[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = ex2(x[e]);
                    f2 w0 = pair(x[0], x[1]), w1 = pair(x[2], x[3]);
                    l2[2 * (i & 1)] = add2(l2[2 * (i & 1)], w0);
                    l2[2 * (i & 1) + 1] = add2(l2[2 * (i & 1) + 1], w1);
                    w0 = mul2(w0, pair(v.x, v.y));
                    w1 = mul2(w1, pair(v.z, v.w));
                    split(w0, x[0], x[1]);
                    split(w1, x[2], x[3]);
                    h[2 * i] = pack2(x[0], x[1]);
                    h[2 * i + 1] = pack2(x[2], x[3]);
                }
                tmem_st_x16(t_s + 16 * c, h);
            }
            if (kTurns<D>) arrive(turn + 8 * (w ^ 1));
            if (rescale) {
                // O is complete up to the step before (its product precedes this S) and no later one has begun
                uint32_t o[D];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tmem_ld_32x32b_x32(t_o + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(o + 32 * c));
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < D; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) tmem_st_x16(t_o + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(o + 16 * c));
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(p_full + 8 * w);
        }
        // the outputs
        float l0, l1;
        split(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])), l0, l1);
        const float l = l0 + l1;
        if (steps > 0 && ok) ok = mbar_wait_warp(o_full, 0, p.status);
        tc_fence_after();
        const int64_t *const place = reinterpret_cast<const int64_t *>(smem_base + S::kOuts) + w * kRows;
        if (p.splits > 1) {
            // the part of the output, by columns so that the rows of a warp lie side by side
            float *const dst = p.part + ((int64_t)item * p.splits + part) * (D + 2) * (2 * kRows) + w * kRows + r;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (steps > 0) {
                    tmem_ld_32x32b_x32(t_o + 32 * c, o);
                    tmem_wait_ld();
                }
                constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};  // dimension of a group's column
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    dst[(32 * c + (i & ~7) + order[i & 7]) * (2 * kRows)] = steps > 0 && ok ? __uint_as_float(o[i]) * (__uint_as_float(vexp) / kSumUnit) : 0.0f;
            }
            dst[D * (2 * kRows)] = ok ? ref : kNone;
            dst[(D + 1) * (2 * kRows)] = ok ? l : 0.0f;
            if (part == 0) p.place[(int64_t)item * (2 * kRows) + w * kRows + r] = place[r];
        } else if (ok) {
            // rows of bf16 over the tile of Q, which no product reads any more; 16-byte pieces swizzled by row
            const float inv = l == 0.0f ? 0.0f : __uint_as_float(vexp) / l;
            constexpr int P = D / 8;  // pieces of a row
            const uint32_t rows_at = base + S::kQ + w * S::kTile + (r & ~31) * P * 16;  // the warp's 32 rows
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (steps > 0) {
                    tmem_ld_32x32b_x32(t_o + 32 * c, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(o[8 * i + e]) * inv;
                    sts128(rows_at + (lane * P + ((4 * c + i) ^ (lane & 7))) * 16, bf2(y[0], y[2]), bf2(y[4], y[6]), bf2(y[1], y[3]), bf2(y[5], y[7]));
                }
            }
            if (p.lse && on) p.lse[place[r]] = l == 0.0f ? -CUDART_INF_F : (ref + log2f(l)) * kLn2;
            __syncwarp();
#pragma unroll 2
            for (int i = 0; i < P; ++i) {
                const int rr = (i * 32 + lane) / P, piece = lane % P;
                uint32_t y[4];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                             : "r"(rows_at + (rr * P + (piece ^ (rr & 7))) * 16)
                             : "memory");
                const int64_t to = place[(r & ~31) + rr];
                if (to >= 0) *reinterpret_cast<uint4 *>(p.out + to * D + 8 * piece) = make_uint4(y[0], y[1], y[2], y[3]);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs<D>));
        const uint32_t magic[2] = {p.magic[0], p.magic[1]};
        auto put_piece = [&](auto keys, uint32_t tile, int i, int q, const uint4 &c) {  // 32 dimensions of position i
            const uint32_t x[4] = {c.x, c.y, c.z, c.w};
            const uint32_t row = tile + (q >> 1) * (kRows * 128) + i * 128;
#pragma unroll
            for (int e = 0; e < 4; ++e) put_codes<decltype(keys)::value>(row + ((((4 * q + e) & 7) ^ (i & 7)) << 4), x[e], magic);
        };
        auto put_bos = [&](auto keys, uint32_t tile, int q, const int8_t *c8) {  // 32 dimensions of position 0, kept at 8 bits
            constexpr float u = decltype(keys)::value ? kKeyUnit : 1.0f;
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
                const char4 a = *reinterpret_cast<const char4 *>(c8 + 32 * q + 8 * e), c = *reinterpret_cast<const char4 *>(c8 + 32 * q + 8 * e + 4);
                sts128(tile + (q >> 1) * (kRows * 128) + (((4 * q + e) & 7) << 4), pack2(a.x * u, c.x * u), pack2(a.y * u, c.y * u),
                       pack2(a.z * u, c.z * u), pack2(a.w * u, c.w * u));
            }
        };
        if (warp < 12) {
            // ------------------------------------------------------------ places, steps and keys
            const int i = tid - 256;  // position within the step
            const uint32_t mask = (1u << p.c.page_log2) - 1;
            auto wanted = [&](int j) {
                const int pos = (step0 + j) * kPos + i;
                return j < steps && pos < end && pos >= begin;
            };
            auto page_of = [&](int j) {
                const int at = ((step0 + j) * kPos + i) >> p.c.page_log2;
                return wanted(j) && at < p.bt.max_pages ? __ldg(p.bt.table + (int64_t)b * p.bt.table_stride + at) : -1;
            };
            // finds the place of this thread's position of step j and tells the others
            auto publish = [&](int j, int page) {
                uint32_t r = kNowhere;
                if (wanted(j)) {
                    if ((unsigned)page < (unsigned)p.c.pages)
                        r = (((uint32_t)page * p.c.heads + kh) << p.c.page_log2) + (((step0 + j) * kPos + i) & mask);
                    else
                        record_status(p.status, (int)BITNET_ERR_INVALID_ARG);
                }
                sts32(base + S::kPlaces + (j % kPlaceStages) * 512 + 4 * i, r);
                arrive(at_full + 8 * (j % kPlaceStages));
                return r;
            };
            uint4 kc[D / 32];
            float ks, vs[4];
            // this position's key codes and step, and the value steps of the positions i % 32 + 32 k
            auto load = [&](int j, uint32_t r) {
                const uint4 *const src = reinterpret_cast<const uint4 *>(p.c.k_codes + (uint64_t)(r == kNowhere ? 0 : r) * (D / 2));
#pragma unroll
                for (int c = 0; c < D / 32; ++c) kc[c] = r != kNowhere ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
                ks = r != kNowhere ? __ldg(p.c.k_step + r) : 0.0f;
                const bool ok = mbar_wait_warp(at_full + 8 * (j % kPlaceStages), (j / kPlaceStages) & 1, p.status);
                const uint32_t places = base + S::kPlaces + (j % kPlaceStages) * 512 + 4 * lane;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t x = lds32(places + 128 * k);
                    vs[k] = x != kNowhere ? __ldg(p.c.v_step + x) : 0.0f;
                }
                return ok;
            };
            uint32_t r = kNowhere, next = kNowhere;
            int page = page_of(1);
            bool ok = true;
            if (steps > 0) {
                r = publish(0, page_of(0));
                next = publish(1, page);
                page = page_of(2);
                ok = load(0, r);
            }
            uint32_t vexp = 0x0d000000u;  // 2^-101
            for (int j = 0; j < steps && ok; ++j) {
                // Slot j + 2 held step j - 6.  This thread has seen k_empty of step j - 3, so the products have seen v_full of
                // step j - 4, after which the value warps read the places of step j - 3 at the earliest.
                const uint32_t after = j + 2 < steps ? publish(j + 2, page) : kNowhere;
                page = page_of(j + 3);
                const bool live = r != kNowhere;
                const uint32_t live_bits = __ballot_sync(0xffffffffu, live);
                uint32_t most = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t bits = __float_as_uint(vs[k]) & 0x7f800000u;
                    most = max(most, bits < 0x7f800000u ? bits : 0u);
                }
                vexp = min(max(vexp, __reduce_max_sync(0xffffffffu, most)), 0x7e000000u);
                const float own = (warp & 2) ? ((warp & 1) ? vs[3] : vs[2]) : ((warp & 1) ? vs[1] : vs[0]);
                // a step that is not finite: NaN for the rows that see it, and for no others (see kv4_rows_kernel)
                const bool bad = !(fabsf(own) < CUDART_INF_F && fabsf(ks) < CUDART_INF_F);
                const int st = j % kStepStages, sk = j % kKS;
                const uint32_t steps_at = base + S::kSteps + st * 1024, meta = base + S::kMeta + st * 32, kt = base + S::kK + sk * S::kTile;
                if (j >= kKS && !mbar_wait_warp(k_empty + 8 * sk, (j / kKS - 1) & 1, p.status)) break;
                sts32(steps_at + 4 * i, __float_as_uint(bad ? CUDART_NAN_F : (live ? ks : 0.0f)));
                sts32(steps_at + 512 + 4 * i, __float_as_uint(bad || !live ? 0.0f : own * __uint_as_float(0x7f000000u - vexp)));
                if (lane == 0) sts32(meta + 4 * (warp - 8), live_bits);
                if (i == 0) sts32(meta + 16, vexp);
                arrive(st_full + 8 * st);
#pragma unroll
                for (int q = 0; q < D / 32; ++q) put_piece(std::true_type(), kt, i, q, kc[q]);
                if (live && (step0 + j) * kPos + i == 0)
                    for (int q = 0; q < D / 32; ++q) put_bos(std::true_type(), kt, q, p.c.k_bos + (int64_t)(r >> p.c.page_log2) * D);
                fence_proxy_async_smem();
                arrive(k_full + 8 * sk);
                if (j + 1 < steps) ok = load(j + 1, next);
                r = next;
                next = after;
            }
        } else if (warp > 12) {
            // ------------------------------------------------------------ values
            const int v = tid - 13 * 32;
            constexpr int kPieces = kPos * D / 32, kRounds = (kPieces + kValueThreads - 1) / kValueThreads;
            uint4 c[kRounds];
            auto load = [&](int j) {  // piece x: 32 dimensions x % (D / 32) of position x / (D / 32)
                if (!mbar_wait_warp(at_full + 8 * (j % kPlaceStages), (j / kPlaceStages) & 1, p.status)) return false;
                const uint32_t places = base + S::kPlaces + (j % kPlaceStages) * 512;
#pragma unroll
                for (int k = 0; k < kRounds; ++k) {
                    const int x = v + k * kValueThreads;
                    const uint32_t r = x < kPieces ? lds32(places + 4 * (x / (D / 32))) : kNowhere;
                    c[k] = r != kNowhere ? __ldg(reinterpret_cast<const uint4 *>(p.c.v_codes + (uint64_t)r * (D / 2)) + x % (D / 32))
                                         : make_uint4(0, 0, 0, 0);
                }
                return true;
            };
            bool ok = steps > 0 && load(0);
            for (int j = 0; j < steps && ok; ++j) {
                const int sv = j % kVS;
                const uint32_t vt = base + S::kV + sv * S::kTile;
                if (j >= kVS && !mbar_wait_warp(v_empty + 8 * sv, (j / kVS - 1) & 1, p.status)) break;
#pragma unroll
                for (int k = 0; k < kRounds; ++k) {
                    const int x = v + k * kValueThreads;
                    if (x < kPieces) put_piece(std::false_type(), vt, x / (D / 32), x % (D / 32), c[k]);
                }
                if (step0 + j == 0 && v < D / 32) {
                    const uint32_t r = lds32(base + S::kPlaces + (j % kPlaceStages) * 512);
                    if (r != kNowhere) put_bos(std::false_type(), vt, v, p.c.v_bos + (int64_t)(r >> p.c.page_log2) * D);
                }
                fence_proxy_async_smem();
                arrive(v_full + 8 * sv);
                if (j + 1 < steps) ok = load(j + 1);
            }
        } else if (warp == 12 && steps > 0) {
            // ------------------------------------------------------------ products
            bool ok = mbar_wait_warp(q_full, 0, p.status);
            const uint64_t q_desc = smem_desc(base + S::kQ, false), k_desc = smem_desc(base + S::kK, false),
                           v_desc = smem_desc(base + S::kV, true);
            constexpr uint32_t id_s = idesc(kPos, false), id_o = idesc(D, true);
            for (int j = 0; j <= steps && ok; ++j) {
                const int sk = j % kKS, sv = (j + kVS - 1) % kVS;  // V of step j - 1
#pragma unroll 1
                for (int w = 0; w < 2; ++w) {
                    if (j > 0) {
                        if (w == 0 && !mbar_wait_warp(v_full + 8 * sv, ((j - 1) / kVS) & 1, p.status)) ok = false;
                        if (!ok || !mbar_wait_warp(p_full + 8 * w, (j - 1) & 1, p.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kPos / 16; ++k)  // 16 positions: 8 columns of P, 16 rows of V
                            mma_ts(tmem + 2 * kPos + w * D, tmem + w * kPos + 8 * k, v_desc + (uint64_t)((sv * S::kTile + k * 2048) >> 4), id_o,
                                   (j > 1 || k > 0) ? 1u : 0u);
                        if (w == 1) umma_commit_elect(v_empty + 8 * sv);
                    }
                    if (j < steps) {
                        if (w == 0 && !mbar_wait_warp(k_full + 8 * sk, (j / kKS) & 1, p.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = (k >> 2) * (kRows * 128) + (k & 3) * 32;
                            mma_ss(tmem + w * kPos, q_desc + (uint64_t)((w * S::kTile + off) >> 4), k_desc + (uint64_t)((sk * S::kTile + off) >> 4),
                                   id_s, k > 0 ? 1u : 0u);
                        }
                        umma_commit_elect(s_full + 8 * w);
                        if (w == 1) umma_commit_elect(k_empty + 8 * sk);
                    }
                }
            }
            // also after a wait that gave up: everything issued ends before the CTA does
            umma_commit_elect(o_full);
            mbar_wait_warp(o_full, 0, p.status);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of 32 rows of an item, in the order of the positions.
template <int D>
__global__ void __launch_bounds__(256) kv4_tiles_join_kernel(const __grid_constant__ TileParams p) {
    __shared__ float out[32][D + 1];
    __shared__ int64_t places[32];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = blockIdx.x >> 3, row = (blockIdx.x & 7) * 32 + lane;
    const float *const src = p.part + (int64_t)item * p.splits * (D + 2) * (2 * kRows) + row;
    constexpr int64_t kPart = (D + 2) * (2 * kRows);
    int64_t place = p.place[(int64_t)item * (2 * kRows) + row];
    if (place >= p.T * p.q_heads) place = -1;  // a workspace that calls share at the same time can hold anything
    if (__syncthreads_and(place < 0)) return;  // nobody's rows, whose parts may not be written
    // everything of a row at a time: the references and sums, then eight parts of four dimensions
    float w[kSplits], l[kSplits], top = kNone, sum = 0.0f;
#pragma unroll
    for (int s = 0; s < kSplits; ++s) {
        w[s] = s < p.splits ? src[s * kPart + D * (2 * kRows)] : kNone;
        l[s] = s < p.splits ? src[s * kPart + (D + 1) * (2 * kRows)] : 0.0f;
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
            for (int s = 0; s < kSplits; ++s) v[e][s] = s < p.splits ? src[s * kPart + (8 * (d0 + e) + warp) * (2 * kRows)] : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y = 0.0f;
#pragma unroll
            for (int s = 0; s < kSplits; ++s) y = fmaf(w[s], v[e][s], y);
            out[lane][8 * (d0 + e) + warp] = y * inv;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * (D / 2); i += 256) {
        const int r = i / (D / 2), d = 2 * (i % (D / 2));
        if (places[r] >= 0)
            *reinterpret_cast<uint32_t *>(p.out + places[r] * D + d) = bf2(out[r][d], out[r][d + 1]);
    }
}

template <int D>
cudaError_t launch_tiles(const TileParams &p, int64_t items, cudaStream_t s) {
    static bool allowed[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !allowed[dev]) {
        e = cudaFuncSetAttribute((const void *)kv4_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
        if (e != cudaSuccess) return e;
        // the softmax warps' registers come out of what the block is launched with
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, (const void *)kv4_tiles_kernel<D>);
        if (e != cudaSuccess) return e;
        if (at.numRegs * kThreads < 256 * (kSoftmaxRegs<D> + kOtherRegs<D>)) return cudaErrorInvalidConfiguration;
        if (dev < kMaxDevices) allowed[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * p.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Smem<D>::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kv4_tiles_kernel<D>, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    cfg.gridDim = dim3((unsigned)(items * 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv4_tiles_join_kernel<D>, p);
}

// The most items (pairs of tiles and key heads) that T rows can make: at most one pair of a sequence is not full.
int64_t most_items(int64_t T, int group, int heads, int batch, int rows_min) {
    const int64_t rows = T * group;
    return (rows / (2 * kRows) + (rows / rows_min < batch ? rows / rows_min : (int64_t)batch)) * heads;
}
// Parts of split items: up to three of them to an SM.
constexpr int kWaves = 3;
int64_t most_splits(int64_t items) {
    const int64_t s = items > 0 ? (int64_t)kWaves * sm_count() / items : 0;
    return s < 1 ? 1 : (s > kSplits ? kSplits : s);
}

}  // namespace

size_t kv4_tiles_workspace(int64_t T, int group, int heads, int dim, int batch, int rows_min) {
    const int64_t items = most_items(T, group, heads, batch, rows_min), splits = most_splits(items);
    if (splits == 1) return 0;
    return (size_t)items * (2 * kRows) * (splits * (dim + 2) * sizeof(float) + sizeof(int64_t));
}

cudaError_t launch_kv4_tiles(const void *q, int64_t T, int q_heads, int64_t qts, int64_t qhs, const Kv4Cache &c,
                             const Kv4Batch &bt, float scale, bool causal, int window, int rows_min, void *out, float *lse,
                             void *ws, cudaStream_t s) {
    TileParams p = {};
    p.q = q, p.qts = qts, p.qhs = qhs, p.q_heads = q_heads, p.group = q_heads / c.heads, p.T = T;
    p.c = c, p.bt = bt, p.scale = scale, p.causal = causal, p.window = window, p.rows_min = rows_min;
    p.out = static_cast<uint16_t *>(out), p.lse = lse, p.status = device_status_ptr();
    p.magic[0] = 0x64086408u, p.magic[1] = 0x64806480u;
    p.by_group = divide_by((uint32_t)p.group);
    const int64_t items = most_items(T, p.group, c.heads, bt.batch, rows_min);
    if (items == 0) return cudaSuccess;
    if (T * p.group > INT32_MAX - 2 * kRows || items * 8 > INT32_MAX) return cudaErrorInvalidConfiguration;
    // With few items the positions are split over several CTAs: as many as leave the SMs least idle, where an
    // item costs as much as kCost steps to begin and to end.  (A chunk of 208 items with 130 steps each on 148 SMs: 522 us
    // unsplit, in two turns of which the second fills two SMs in five, and 456 us split; 700 tokens of one head of dim 128:
    // 31 and 28.)  Joining costs about a step.
    constexpr int kCost = 6, kJoin = 1;
    const int64_t steps = ceil_div((int64_t)bt.max_pages << c.page_log2, kPos), sms = sm_count();
    int64_t best = -1;
    p.splits = 1;
    for (int64_t n = 1; n <= most_splits(items) && (n == 1 || steps >= 2 * n); ++n) {
        const int64_t cost = ceil_div(items * n, sms) * (kCost + ceil_div(steps, n)) + (n > 1 ? kJoin : 0);
        if (best < 0 || cost < best) best = cost, p.splits = (int)n;
    }
    p.place = static_cast<int64_t *>(ws);
    p.part = reinterpret_cast<float *>(p.place + items * (2 * kRows));
    return c.dim == 64 ? launch_tiles<64>(p, items, s) : launch_tiles<128>(p, items, s);
}

}  // namespace bitnet
