// kv4_attention.cu -- softmax attention over the 4-bit paged KV cache.
//
// Method: bitnet_v2_engine.py page, BitNetV2Attention.forward on the fake-quantised keys and
// values: s_t = scale * kstep_t * (q . kcode_t), out = sum_t e^(s_t) vstep_t vcode_t / sum_t e^(s_t).
//
// Few rows to a sequence (decode, draft tokens): kv4_rows_kernel, below.  A sequence's rows
// that share a key head (new tokens x query heads of the group) are one item of 8 * NT rows;
// codes pass from memory to registers once and become fp16 operands of mma.sync there, with
// the positions as the 16-side and the rows as the 8-side of the product, so that nothing is
// padded for groups of up to 8.
//
// What bounds it: 64 sequences of 256 to 8192 positions, 32 query heads on 8 of dim 128, one new
// token each (296 MB of cache): 85 us, 3.5 TB/s; two of 131072 and 111869 positions with 64 query heads:
// 71 us, 3.7 TB/s.  Without its arithmetic the kernel took 70 and 53 us of 84 and 70: a tile costs a warp 620 instructions
// (300 of them turn nibbles into fp16 and 32 are products), which keeps 61 % of the issue slots and half of the
// integer units busy, and an item's beginning and end take as long as 16 tiles of its CTA.  fp32 calls double
// the products: 4 sequences of 4096 positions, 32 heads each with its own keys, 34 us.  Tried, and no
// faster: bulk copies (107 us where these took 99), four CTAs to an SM, codes as subnormal fp16 (2 % at the cost
// of small weights' bits).
#include "kv4.cuh"

#include <cuda_fp16.h>
#include <math_constants.h>

namespace bitnet {

namespace {

constexpr int kWarps = 4;
constexpr uint32_t kNowhere = 0xffffffffu;
constexpr int kTile = 32;       // positions that a warp takes at a time
constexpr int kMaxParts = 64;   // CTAs that may share an item on average
constexpr int kMinTiles = 4;    // tiles that make a CTA of its own worth while
constexpr int kJoinSplit = 2;   // CTAs that join an item, each some of its rows
// Items that can have no more tiles than this are not shared between CTAs (then there is nothing to join), and twice as
// many where there are items for every other SM.  Measured in a graph (whole, shared) at 8 key heads of dim 128: 64
// sequences of 500 positions 27 and 33 us; 32, 16, 8 and 4 of 1000 positions 21 and 28, 19 and 21, 18 and 18, 18 and
// 15; one of 1000 15 and 9.  One of 500 is 11 and 9, but the call takes 13.8 and 17.8, which the host's second launch bounds.
constexpr int kWholeTiles = 18;
constexpr int kItemCost = 16;   // what beginning and ending an item takes, in tiles
// Weights are held as 2^(s - m + kOff), and a score may pass the running maximum m by kLag before
// that moves: with a step ratio below 2 they stay below 2^15.  The more below, the more references move and the finer the
// smallest weights are: with 2^3 and 11 for bf16 calls these lost three bits for 1 % of the time (64 sequences of 256 to 8192
// positions 84.3 us instead of 84.9).  fp32 calls leave less room above, for a finer second part.
template <bool BF16>
constexpr float kOff = BF16 ? 6.0f : 13.0f;
template <bool BF16>
constexpr float kLag = BF16 ? 8.0f : 1.0f;
constexpr float kNone = -3.0e38f;  // reference (m - kOff) of a row that has seen nothing yet
constexpr int kTilesFrom = 128;  // rows of a sequence from which on kv4_prefill.cu or kv4_chunk.cu takes them
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int N>
struct Const {
    __host__ __device__ constexpr operator int() const { return N; }
};
template <int N, typename F>
__device__ __forceinline__ void each(F f) {  // f(constant 0), ..., f(constant N - 1)
    if constexpr (N > 0) {
        each<N - 1>(f);
        f(Const<N - 1>());
    }
}

// A stage of a warp's ring: a tile's keys, values and steps, copied 16 bytes a lane as they lie
// in the cache, but for an order of the chunks in which the lanes' loads meet no bank twice.
// Lane (g, t) loads D / 8 bytes of key rows rk(g) + 8 n, rk = 4 (g % 2) + g / 2, at t, and D / 16
// bytes of value rows t + 4 n at g.
template <int D>
struct Ring {
    static constexpr uint32_t kRow = D / 2, kChunks = D / 32, kBlock = 16 * kRow;  // a row, its chunks, a block of 16
    static constexpr uint32_t kKeys = 0, kValues = 2 * kBlock, kSteps = 4 * kBlock;
    static constexpr uint32_t kStage = kSteps + 2 * 4 * kTile;
    // chunk c of row r, for the rows of a copy (of 512 / kRow rows)
    static __device__ __forceinline__ uint32_t key(uint32_t r, uint32_t c) {
        if constexpr (D == 64) return (r ^ (r >> 1 & 2)) * kRow + c * 16;
        if constexpr (D == 128) return (r ^ (r >> 2 & 1)) * kRow + c * 16;
        return r * kRow + (c ^ (r >> 2 & 1)) * 16;
    }
    static __device__ __forceinline__ uint32_t value(uint32_t r, uint32_t c) {
        if constexpr (D == 64) return r * kRow + c * 16;
        if constexpr (D == 128) return r * kRow + (c ^ (r & 2)) * 16;
        return r * kRow + (c ^ (r & 3) * 2) * 16;
    }
};
// Tiles of a warp under way at a time: what fits the shared memory of an SM with kResident CTAs.
// CTAs of an SM: three where their registers allow it (bf16, dim 128, 8 rows: 84 us for 64 sequences
// of 256 to 8192 positions, against 88 with two).
template <int D, int NT, bool BF16>
constexpr int kResident = NT == 1 && (D == 64 || (D == 128 && BF16)) ? 3 : 2;
template <int D, int NT, bool BF16>
constexpr int kStages = D == 256 ? 3 : (D / 64 * kResident<D, NT, BF16> == 6 ? 4 : 5);
template <int D, int NT, bool BF16>
constexpr int kRowsSmem = kWarps * ((int)(kStages<D, NT, BF16> * Ring<D>::kStage) > 8 * NT * (D + 4) * 4 ? (int)(kStages<D, NT, BF16> * Ring<D>::kStage)
                                                                                                        : 8 * NT * (D + 4) * 4);

struct RowsParams {
    const void *q;
    int64_t qts, qhs;
    int q_heads, group;  // query heads, and those of one key head
    int64_t T;
    Kv4Cache c;
    Kv4Batch bt;
    float scale;
    int causal;
    int window;   // INT32_MAX: none
    int whole;    // every item is one CTA's, and there is no kernel to join parts
    int rows_max; // sequences with more rows (new tokens x group) are another kernel's
    void *out;
    float *lse;
    float *part;  // [grid][2]: outputs [8 NT][D], then reference and sum [8 NT][2]
    int4 *head;   // [grid]: where this CTA's first part is the second of its item, {the sequence's first row among the
                  // call's, the item's first row, its rows + 256 * key head, its parts}; no parts otherwise
    int *status;
    uint32_t magic[2];  // see halves()
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with nothing to add to.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t h2_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ uint32_t h2(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// Nibbles (0, 4), (1, 5), (2, 6), (3, 7) of a word as pairs of codes in fp16: (n ^ 8) = code + 8 goes into
// the mantissa of 1024, which is then taken off (for the odd nibbles, which stand four bits
// higher, with a factor 1/16).  magic is {0x64086408, 0x64806480}, in registers: a logic
// instruction takes one constant, so that with two of them each half would cost two (measured: 291
// to a tile instead of 165, on the pipe that binds).
__device__ __forceinline__ void halves(uint32_t w, const uint32_t (&magic)[2], uint32_t (&h)[4]) {
    const uint32_t v = w >> 8;
    const __half2 off = __float2half2_rn(-1032.0f), off16 = __float2half2_rn(-72.0f), sixteenth = __float2half2_rn(0.0625f);
    h[0] = h2(__hadd2(as_h2((w & 0x000F000Fu) ^ magic[0]), off));
    h[1] = h2(__hfma2(as_h2((w & 0x00F000F0u) ^ magic[1]), sixteenth, off16));
    h[2] = h2(__hadd2(as_h2((v & 0x000F000Fu) ^ magic[0]), off));
    h[3] = h2(__hfma2(as_h2((v & 0x00F000F0u) ^ magic[1]), sixteenth, off16));
}

// A lane's copy of 16 bytes into shared memory; zeros where !on (nothing is read then).
template <int TO, int FROM>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t on) {
    asm volatile("{.reg .pred p; setp.eq.u32 p, %2, 0; cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16, p;}" ::"r"(dst),
                 "l"(src), "r"(on), "n"(TO), "n"(FROM)
                 : "memory");
}
// BYTES (4, 8 or 16) from shared memory.
template <int BYTES, int FROM>
__device__ __forceinline__ void take(uint32_t src, uint32_t *w) {
    if constexpr (BYTES == 4) {
        asm volatile("ld.shared.b32 %0, [%1 + %2];" : "=r"(w[0]) : "r"(src), "n"(FROM) : "memory");
    } else if constexpr (BYTES == 8) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2 + %3];" : "=r"(w[0]), "=r"(w[1]) : "r"(src), "n"(FROM) : "memory");
    } else {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(src), "n"(FROM)
                     : "memory");
    }
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// A sequence's items: row tiles of R rows, and the tiles of positions that each may need.
struct Seq {
    int first;  // its first row among the call's
    int base;   // position of that row
    int cap;    // positions that the cache can hold of it
    int rows, row_tiles, tiles;
};
template <int R>
__device__ __forceinline__ Seq seq_of(const RowsParams &p, int b) {
    Seq s;
    s.first = max(0, __ldg(p.bt.starts + b));
    const int n = max(0, __ldg(p.bt.starts + b + 1) - s.first);
    const int len = max(0, __ldg(p.bt.lens + b));
    s.base = len - n;
    s.cap = (int)min((int64_t)len, (int64_t)p.bt.max_pages << p.c.page_log2);
    // rows past the end of the tensors are nobody's
    const int64_t rows = (int64_t)min((int64_t)n, max((int64_t)0, p.T - s.first)) * p.group;
    s.rows = rows > p.rows_max ? 0 : (int)rows;
    s.row_tiles = (s.rows + R - 1) / R;
    // a row tile stands on at most R / group + 2 tokens
    const int64_t span = min((int64_t)s.cap, (int64_t)p.window + R / p.group + 2);
    s.tiles = max(1, (int)((span + kTile - 1) / kTile) + (p.window < len ? 1 : 0));
    if (s.cap < len && s.rows > 0) record_status(p.status, (int)BITNET_ERR_INVALID_ARG);
    return s;
}
__device__ __forceinline__ int unit_of(const RowsParams &p, const Seq &s) { return p.whole ? 1 : s.tiles + kItemCost; }
__device__ __forceinline__ int64_t weight(const RowsParams &p, const Seq &s) {
    return (int64_t)s.row_tiles * p.c.heads * unit_of(p, s);
}

// Every CTA takes an equal run of all tiles of all items, in order; the run's first and last
// item may be shared with its neighbours.  Their parts (output, reference, sum) go to the
// workspace and kv4_join_kernel adds them up, in the order of the positions.
//
// Of a tile a warp computes S = K Q^T (positions x rows) with keys as the left operand, turns
// the weights' 8 x 8 blocks with movmatrix into the right operand of O = V^T P
// (dimensions x rows), whose left operand takes two positions' codes to a register.  Lane (g, t) =
// (lane / 4, lane % 4) holds position 4 (g % 2) + g / 2 (+ 8) of a block of 16 as row g (+ 8),
// so that the positions t, t + 4, t + 8, t + 12, which it needs of the values, lie in
// neighbouring rows of the cache over t.
//
// Scores stand in units of log2.  The running maximum m of a row moves only when a score
// passes it by more than kLag, so most tiles have no reduction and no rescaling; weights
// 2^(s - m + kOff) stay below 2^15 and keep fp16's eleven bits down to 2^-20 of the maximum.
// A tile's value steps are divided by a power of two that none is twice as large as, which scales the
// tile's product in fp32.  (With O in the products' own registers, in units of the largest step so far, two long sequences
// took 1 % less; positions behind a far larger step lost their bits.)
// Queries are scaled by a power of two into [2^14, 2^15); bf16 queries are then exact in
// fp16 down to 2^-28 of the row's maximum.  fp32 calls carry queries and weights as the
// sum of two fp16 numbers (22 bits).
template <int D, int NT, bool BF16>
__global__ void __launch_bounds__(32 * kWarps, kResident<D, NT, BF16>)
kv4_rows_kernel(const __grid_constant__ RowsParams p) {
    constexpr int R = 8 * NT;
    constexpr int KW = D / 32;  // words of keys per lane and position
    constexpr int VW = D / 64;  // words of values per lane and position
    constexpr int NP = BF16 ? 1 : 2;
    constexpr int LD = D + 4;
    extern __shared__ __align__(128) float so[];  // [kWarps][R][LD] once the loop is done, the warps' rings before
    __shared__ float sm[kWarps][R], sl[kWarps][R];
    __shared__ int64_t scan[2 * kWarps];
    __shared__ int start_b;
    __shared__ int64_t start_off;

    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(so) + warp * (kStages<D, NT, BF16> * Ring<D>::kStage);
    const int B = p.bt.batch;
    const uint32_t magic[2] = {p.magic[0], p.magic[1]};

    // this CTA's run [run, run_end) of the W tiles
    const int per = (B + 32 * kWarps - 1) / (32 * kWarps);
    int64_t mine = 0;
    int64_t items = 0;
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) {
        const Seq s = seq_of<R>(p, b);
        mine += weight(p, s);
        items += (int64_t)s.row_tiles * p.c.heads;
    }
    int64_t before = mine, all_items = items;  // inclusive sums over the warp, then over the CTA
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, before, x);
        if (lane >= x) before += y;
        all_items += __shfl_xor_sync(0xffffffffu, all_items, x);
    }
    if (lane == 31) scan[warp] = before;
    if (lane == 0) scan[kWarps + warp] = all_items;
    __syncthreads();
    int64_t W = 0;
    items = 0;
    before -= mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? scan[w] : 0;
        W += scan[w];
        items += scan[kWarps + w];
    }
    int64_t G = gridDim.x;
    G = max((int64_t)1, p.whole ? min(G, W) : min(min(G, items * kMaxParts), (W + kMinTiles - 1) / kMinTiles));
    const int64_t cta = blockIdx.x;
    const int64_t run0 = cta < G ? W * cta / G : W, run_end = cta < G ? W * (cta + 1) / G : W;
    if (run0 >= run_end) {
        if (tid == 0) p.head[cta] = make_int4(0, 0, 0, 0);
        return;
    }
    if (run0 >= before && run0 < before + mine) {
        int b = tid * per;
        int64_t off = run0 - before;
        while (true) {
            const int64_t w = weight(p, seq_of<R>(p, b));
            if (off < w) break;
            off -= w;
            ++b;
        }
        start_b = b;
        start_off = off;
    }
    __syncthreads();
    int b = start_b;
    int64_t off = start_off;

    int64_t run = run0;
    while (run < run_end) {
        Seq s = seq_of<R>(p, b);
        while (off >= weight(p, s)) {  // the next sequence with items
            off -= weight(p, s);
            s = seq_of<R>(p, ++b);
        }
        const int unit = unit_of(p, s);
        const int item = (int)(off / unit);  // key head * row tiles + row tile
        const int kh = item / s.row_tiles, rt = item - kh * s.row_tiles;
        const int from = (int)(off - (int64_t)item * unit), to = (int)min((int64_t)unit, from + (run_end - run));
        const bool starts = from == 0, whole = starts && to == unit;
        const int lo = p.whole ? 0 : max(0, from - kItemCost), hi = p.whole ? s.tiles : max(0, to - kItemCost);  // tiles
        if (run == run0 && tid == 0) {
            // where this CTA's first part is the second of its item, it names the CTAs that share the item
            int4 h = make_int4(0, 0, 0, 0);
            const int64_t first = run0 - from;  // of the item
            if (!starts && W * (cta - 1) / G <= first) {
                const int64_t last = ((first + unit) * G + W - 1) / W - 1;  // the first whose run ends behind the item
                h = make_int4(s.first, rt * R, min(R, s.rows - rt * R) + 256 * kh, (int)(last - cta + 2));
            }
            p.head[cta] = h;
        }
        const int row0 = rt * R, nrows = min(R, s.rows - row0);
        const int q0 = s.first, base = s.base;
        const int tok0 = row0 / p.group, tok1 = (row0 + nrows - 1) / p.group;
        // positions that some row of the tile sees, and those that all see
        const int end = p.causal ? min(s.cap, base + tok1 + 1) : s.cap;
        const int begin = (int)max((int64_t)0, (int64_t)base + tok0 - p.window + 1) * p.causal;
        const int all_end = p.causal ? base + tok0 + 1 : s.cap;
        const int all_begin = p.causal ? (int)max((int64_t)0, (int64_t)base + tok1 - p.window + 1) : 0;
        const int tile0 = begin / kTile;
        // position 0 is kept at 8 bits: the item's first warp begins with it, and no tile has it
        const int bos_page = starts && warp == 0 && begin == 0 && end > 0 ? kv4_page(p.c, p.bt, b, 0, p.status) : -1;

        // The warp's tiles lo + warp, + kWarps, ...: their blocks of 16 positions lie in the cache from these
        // rows on, or kNowhere where no page holds them or nothing in them is seen.  Lane 2 i + h has half h
        // of tile 16 n + i; the next 16 tiles' page numbers are on their way meanwhile.
        const uint32_t mask = (1u << p.c.page_log2) - 1;
        const int count = max(0, (min(hi, (end - tile0 * kTile + kTile - 1) / kTile) - lo - warp + kWarps - 1) / kWarps);
        auto block_at = [&](int i) { return (tile0 + lo + warp + (i + (lane >> 1)) * kWarps) * kTile + 16 * (lane & 1); };
        auto wanted = [&](int i) {
            const int at = block_at(i);
            return i + (lane >> 1) < count && at < end && at + 16 > begin;
        };
        auto page_of = [&](int i) {
            const int n = block_at(i) >> p.c.page_log2;
            return wanted(i) && n < p.bt.max_pages ? __ldg(p.bt.table + (int64_t)b * p.bt.table_stride + n) : -1;
        };
        auto rows_of = [&](int i, int page) {
            if (!wanted(i)) return kNowhere;
            if ((unsigned)page >= (unsigned)p.c.pages) {
                record_status(p.status, (int)BITNET_ERR_INVALID_ARG);
                return kNowhere;
            }
            return (((uint32_t)page * p.c.heads + kh) << p.c.page_log2) + (block_at(i) & mask);
        };
        const int page0 = page_of(0);
        int pages = page_of(16);
        // the queries are on their way with the page numbers
        constexpr int QV = D / 4 / (BF16 ? 8 : 4);
        uint4 raw[NT][QV];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = row0 + 8 * nt + g, tok = r / p.group;
            const bool on = 8 * nt + g < nrows;
            const int64_t at = on ? (int64_t)(q0 + tok) * p.qts + (int64_t)(kh * p.group + r - tok * p.group) * p.qhs + t * (D / 4) : 0;
            const uint4 *const src = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(p.q) + at * (BF16 ? 2 : 4));
#pragma unroll
            for (int i = 0; i < QV; ++i) raw[nt][i] = on ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        }
        uint32_t rows = rows_of(0, page0);

        const int rk = 4 * (g & 1) + (g >> 1);
        using S = Ring<D>;
        const uint32_t row_in = lane / S::kChunks, chunk_in = lane % S::kChunks;
        const uint32_t key_in = S::kKeys + S::key(row_in, chunk_in), value_in = S::kValues + S::value(row_in, chunk_in);
        const uint8_t *const k_base = p.c.k_codes + lane * 16, *const v_base = p.c.v_codes + lane * 16;
        const float *const step_base = (lane & 8 ? p.c.v_step : p.c.k_step) + (lane & 3) * 4;
        uint32_t valid = 0;  // two bits for each tile under way: whether its blocks lie somewhere
        auto fetch = [&](int i, uint32_t slot) {  // the copies of the warp's tile i; one group, empty past the end
            valid <<= 2;
            if (i < count) {
                if ((i & 15) == 0 && i > 0) {
                    rows = rows_of(i, pages);
                    pages = page_of(i + 16);
                }
                uint32_t r[2];
                const uint32_t to_k = slot + key_in, to_v = slot + value_in;
                each<2>([&](auto h) {
                    r[h] = __shfl_sync(0xffffffffu, rows, 2 * (i & 15) + h);
                    const uint32_t on = r[h] != kNowhere;
                    valid |= on << h;
                    const uint64_t off = (uint64_t)(on ? r[h] : 0) * S::kRow;
                    const uint8_t *const k = k_base + off, *const v = v_base + off;
                    each<D / 64>([&](auto e) {
                        // of dim 256, every other copy has the rows 4 .. 7 of 8
                        copy_async<h * S::kBlock + e * 512, e * 512>(D == 256 && (e & 1) ? to_k ^ 16 : to_k, k, on);
                        copy_async<h * S::kBlock + e * 512, e * 512>(to_v, v, on);
                    });
                });
                // lanes 0 .. 7 bring the key steps, 8 .. 15 the value steps
                const uint32_t own = lane & 4 ? r[1] : r[0];
                const uint32_t on = own != kNowhere;
                if (lane < 16) copy_async<S::kSteps, 0>(slot + lane * 16, step_base + (on ? own : 0), on);
            }
            copies_commit();
        };
        const uint32_t key_out = S::kKeys + S::key(rk, t * (D / 8) / 16) + t * (D / 8) % 16;
        const uint32_t value_out = S::kValues + S::value(t, g * (D / 16) / 16) + g * (D / 16) % 16;
        uint32_t slot_in = ring, slot_out = ring;
        auto advance = [&](uint32_t &slot) {
            slot += Ring<D>::kStage;
            if (slot == ring + kStages<D, NT, BF16> * Ring<D>::kStage) slot = ring;
        };
#pragma unroll
        for (int i = 0; i < kStages<D, NT, BF16> - 1; ++i) {
            fetch(i, slot_in);
            advance(slot_in);
        }
        // queries: row 8 nt + g, dimensions t D/4 ...; factor and reference for the rows 2t, 2t + 1
        uint32_t qf[NT][NP][KW][2][2];
        float factor[NT][2], ref[NT][2];
        int pos[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[D / 4], top = 0.0f;
#pragma unroll
            for (int i = 0; i < QV; ++i) {
                const uint32_t w[4] = {raw[nt][i].x, raw[nt][i].y, raw[nt][i].z, raw[nt][i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (BF16) {
                        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                    } else {
                        x[4 * i + j] = __uint_as_float(w[j]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // up = 2^(14 - exponent), kept inside the normal numbers (a row below 2^-112 is then scaled less)
            const uint32_t up_bits = min(max(0x86000000u - (__float_as_uint(top) & 0x7f800000u), 0x07000000u), 0x7e800000u);
            const float up = top > 0.0f ? __uint_as_float(up_bits) : 1.0f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) x[i] *= up;
            // of row n in lanes 4 n ...; an infinite query is NaN, as scores of one sign alone would hide every position
            const float f = top < CUDART_INF_F ? p.scale * kLog2e * (1.0f / up) : CUDART_NAN_F;
            float z0 = 0.0f;  // this row's product with position 0
            if (bos_page >= 0) {
                const int8_t *c8 = p.c.k_bos + ((int64_t)bos_page * p.c.heads + kh) * D + t * (D / 4);
#pragma unroll
                for (int i = 0; i < D / 4; i += 4) {
                    const char4 u = *reinterpret_cast<const char4 *>(c8 + i);
                    z0 = fmaf(x[i], u.x, z0), z0 = fmaf(x[i + 1], u.y, z0);
                    z0 = fmaf(x[i + 2], u.z, z0), z0 = fmaf(x[i + 3], u.w, z0);
                }
                z0 += __shfl_xor_sync(0xffffffffu, z0, 1);
                z0 += __shfl_xor_sync(0xffffffffu, z0, 2);
                z0 *= f * p.c.k_step[kv4_rows(p.c, bos_page, kh)];
            }
#pragma unroll
            for (int j = 0; j < KW; ++j)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {  // product m takes nibbles m, m + 4 and m + 2, m + 6
                        const float y0 = x[8 * j + m + 2 * e], y1 = x[8 * j + m + 2 * e + 4];
                        qf[nt][0][j][m][e] = pack2(y0, y1);
                        if constexpr (!BF16)
                            qf[nt][NP - 1][j][m][e] = pack2(y0 - __half2float(__float2half_rn(y0)), y1 - __half2float(__float2half_rn(y1)));
                    }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                factor[nt][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + e));
                pos[nt][e] = base + (row0 + 8 * nt + 2 * t + e) / p.group;
                const float z = __shfl_sync(0xffffffffu, z0, 4 * (2 * t + e));
                const bool sees = bos_page >= 0 && (!p.causal || (pos[nt][e] >= 0 && pos[nt][e] < p.window));
                ref[nt][e] = sees ? z - kOff<BF16> + (z - z) : kNone;  // an infinite score gives NaN
            }
        }

        float l[NT][2], o[NT][D / 16][4];
        const float bos_step = bos_page >= 0 ? p.c.v_step[kv4_rows(p.c, bos_page, kh)] : 0.0f;
        const bool bos_bad = !(fabsf(bos_step) < CUDART_INF_F);  // as for the other positions: NaN for the rows that see it
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float w = ref[nt][c] == kNone ? 0.0f : (bos_bad ? CUDART_NAN_F : (BF16 ? 0x1p6f : 0x1p13f));
                l[nt][c] = g == 0 ? w : 0.0f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) o[nt][i][c] = o[nt][i][2 + c] = w == 0.0f ? 0.0f : w / kSumUnit * bos_step;
            }
        if (bos_page >= 0) {
            const int8_t *c8 = p.c.v_bos + ((int64_t)bos_page * p.c.heads + kh) * D + g * (D / 8);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const int d = 8 * (i >> 2) + 4 * ((i >> 1) & 1) + (i & 1);
                const float x = (float)c8[d], y = (float)c8[d + 2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) o[nt][i][0] *= x, o[nt][i][1] *= x, o[nt][i][2] *= y, o[nt][i][3] *= y;
            }
        }

        for (int it = 0; it < count; ++it) {
            const int at = (tile0 + lo + warp + it * kWarps) * kTile;
            fetch(it + kStages<D, NT, BF16> - 1, slot_in);
            advance(slot_in);
            copies_wait<kStages<D, NT, BF16> - 1>();
            __syncwarp();  // a lane waits for its own copies; it reads the others' too

            // S = K Q^T
            float sc[NT][2][4];
            const uint32_t from_k = slot_out + key_out, from_v = slot_out + value_out;
            each<2>([&](auto h) {
                uint32_t kw[2][KW];
                each<2>([&](auto e) {
                    take<(D < 256 ? D / 8 : 16), h * S::kBlock + 8 * e * S::kRow>(from_k, kw[e]);
                    if constexpr (D == 256) take<16, h * S::kBlock + 8 * e * S::kRow>(from_k ^ 16, kw[e] + 4);
                });
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    uint32_t x[4], y[4];
                    halves(kw[0][j], magic, x);
                    halves(kw[1][j], magic, y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k2 = NP - 1; k2 >= 0; --k2) {
                            if (j == 0 && k2 == NP - 1)
                                mma_f16_first(sc[nt][h], x[0], y[0], x[2], y[2], qf[nt][k2][j][0][0], qf[nt][k2][j][0][1]);
                            else
                                mma_f16(sc[nt][h], x[0], y[0], x[2], y[2], qf[nt][k2][j][0][0], qf[nt][k2][j][0][1]);
                            mma_f16(sc[nt][h], x[1], y[1], x[3], y[3], qf[nt][k2][j][1][0], qf[nt][k2][j][1][1]);
                        }
                }
            });
            // the lane's own position: its key step, and its value step over a power of two that
            // no step of the tile is twice as large as
            const int own = at + lane;
            uint32_t steps[2];
            take<4, S::kSteps>(slot_out + lane * 4, &steps[0]);
            take<4, S::kSteps + 4 * kTile>(slot_out + lane * 4, &steps[1]);
            const bool live = own >= max(begin, 1) && own < end && (valid >> (2 * (kStages<D, NT, BF16> - 1) + (lane >> 4)) & 1);
            const uint32_t vbits = live ? steps[1] & 0x7f800000u : 0u;
            // a step that is not finite: NaN for the rows that see it, and for no others (an infinite key step would turn a
            // negative product into the score that hides a position)
            const bool bad = live && max(vbits, steps[0] & 0x7f800000u) == 0x7f800000u;
            const float kstep = bad ? CUDART_NAN_F : (live ? __uint_as_float(steps[0]) : 0.0f);
            const float vstep = live && !bad ? __uint_as_float(steps[1]) : 0.0f;
            const uint32_t live_bits = __ballot_sync(0xffffffffu, live);
            const uint32_t vexp = min(max(__reduce_max_sync(0xffffffffu, bad ? 0u : vbits), 0x0d000000u), 0x7e000000u);
            const float vtop = __uint_as_float(vexp) / kSumUnit;
            const float vrel = vstep * __uint_as_float(0x7f000000u - vexp);
            const bool edge = at < all_begin || at + kTile > all_end || live_bits != 0xffffffffu;

            // scores less the reference; where one is too far above it, the references move first
            float st[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) st[i] = __shfl_sync(0xffffffffu, kstep, 8 * i + rk);
            float y[NT][8];  // element i: position 8 (i / 2) + rk of the tile, row 2 t + i % 2
            auto hide = [&](float(&z)[NT][8]) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = 8 * (i >> 1) + rk, s = at + j;
                        const bool sees = (live_bits >> j & 1) && (!p.causal || (s <= pos[nt][i & 1] && pos[nt][i & 1] - s < p.window));
                        if (!sees) z[nt][i] = -CUDART_INF_F;
                    }
            };
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[nt][i] = fmaf(sc[nt][i >> 2][i & 3], st[i >> 1] * factor[nt][i & 1], -ref[nt][i & 1]);
                if (edge) hide(y);
                float top = y[0][0];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, y[nt][i]);
                if (pass == 1 || !__any_sync(0xffffffffu, top > kOff<BF16> + kLag<BF16>)) break;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float most = -CUDART_INF_F;
#pragma unroll
                        for (int i = c; i < 8; i += 2)
                            if (y[nt][i] != -CUDART_INF_F) most = fmaxf(most, sc[nt][i >> 2][i & 3] * (st[i >> 1] * factor[nt][c]));
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
                        // only the rows that ask for it, so that a row does not depend on its neighbours
                        most = most - ref[nt][c] > kOff<BF16> + kLag<BF16> ? most - kOff<BF16> : ref[nt][c];
                        const float a = ex2(ref[nt][c] - most);
                        ref[nt][c] = most;
                        l[nt][c] *= a;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) o[nt][i][c] *= a, o[nt][i][2 + c] *= a;
                    }
            }
            // weights, times the values' steps, as the right operand
            uint32_t pf[NT][NP][2][2];
            float vr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[i] = __shfl_sync(0xffffffffu, vrel, 8 * i + rk);
            float w[NT][8];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    w[nt][i] = ex2(y[nt][i]);
                    l[nt][i & 1] += w[nt][i];
                    w[nt][i] *= vr[i >> 1];
                }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t hi2 = pack2(w[nt][2 * i], w[nt][2 * i + 1]);
                    pf[nt][0][i >> 1][i & 1] = transpose8(hi2);
                    if constexpr (!BF16) {
                        const float2 f2 = __half22float2(as_h2(hi2));
                        pf[nt][NP - 1][i >> 1][i & 1] = transpose8(pack2(w[nt][2 * i] - f2.x, w[nt][2 * i + 1] - f2.y));
                    }
                }
            // O = O + V^T P
            uint32_t vw[8][VW];
            each<8>([&](auto i) { take<D / 16, 4 * i * S::kRow>(from_v, vw[i]); });
            __syncwarp();  // the last reads of this stage, which the next fetch() fills again
#pragma unroll
            for (int j = 0; j < VW; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) {  // nibbles 0 .. 3 or 4 .. 7 of the word
                    uint32_t x[2][2][4];       // [block][positions t, t + 4 or t + 8, t + 12][nibble]
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            halves(__byte_perm(vw[4 * h + 2 * e][j], vw[4 * h + 2 * e + 1][j], u ? 0x7632 : 0x5410), magic, x[h][e]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd) {
                            float(&dst)[4] = o[nt][4 * j + 2 * u + odd];
                            // the tensor cores' sums are cut short: they end with the tile
                            float acc[4];
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int k2 = NP - 1; k2 >= 0; --k2) {
                                    if (h == 0 && k2 == NP - 1)
                                        mma_f16_first(acc, x[h][0][odd], x[h][0][odd + 2], x[h][1][odd], x[h][1][odd + 2],
                                                      pf[nt][k2][h][0], pf[nt][k2][h][1]);
                                    else
                                        mma_f16(acc, x[h][0][odd], x[h][0][odd + 2], x[h][1][odd], x[h][1][odd + 2], pf[nt][k2][h][0],
                                                pf[nt][k2][h][1]);
                                }
#pragma unroll
                            for (int i = 0; i < 4; ++i) dst[i] = fmaf(vtop, acc[i], dst[i]);
                        }
                }
            advance(slot_out);
        }
        copies_wait<0>();
        __syncthreads();  // every warp is done with its ring

        // join the warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
                const int n = 8 * nt + 2 * t + c;
                if (g == 0) sm[warp][n] = ref[nt][c], sl[warp][n] = l[nt][c];
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int d = g * (D / 8) + 8 * (i >> 2) + 4 * ((i >> 1) & 1) + (i & 1);
                    so[(warp * R + n) * LD + d] = o[nt][i][c];
                    so[(warp * R + n) * LD + d + 2] = o[nt][i][2 + c];
                }
            }
        __syncthreads();
        float *part = p.part + ((cta * 2 + (starts ? 1 : 0)) * R) * (D + 2);
        for (int i = tid; i < nrows * (D / 4); i += 32 * kWarps) {
            const int n = i / (D / 4), d = 4 * (i % (D / 4));
            float top = kNone, sum = 0.0f;
            float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w][n]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(sm[w][n] - top);
                const float4 x = *reinterpret_cast<const float4 *>(so + (w * R + n) * LD + d);
                sum = fmaf(f, sl[w][n], sum);
                y.x = fmaf(f, x.x, y.x), y.y = fmaf(f, x.y, y.y), y.z = fmaf(f, x.z, y.z), y.w = fmaf(f, x.w, y.w);
            }
            if (!whole) {
                *reinterpret_cast<float4 *>(part + n * D + d) = y;
                if (d == 0) *reinterpret_cast<float2 *>(part + R * D + 2 * n) = make_float2(top, sum);
                continue;
            }
            const int r = row0 + n, tok = r / p.group;
            const int64_t at = (int64_t)(q0 + tok) * p.q_heads + kh * p.group + (r - tok * p.group);
            const float inv = sum == 0.0f ? 0.0f : kSumUnit / sum;
            if constexpr (BF16)
                *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p.out) + at * D + d) = make_uint2(
                    h2_bf16(y.x * inv, y.y * inv), h2_bf16(y.z * inv, y.w * inv));
            else
                *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.out) + at * D + d) =
                    make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
            if (p.lse && d == 0) p.lse[at] = sum == 0.0f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2;
        }
        __syncthreads();
        run += to - from;
        off += to - from;
    }
}

// Joins the parts of the items that several CTAs of kv4_rows_kernel shared: one CTA to each of
// that kernel's, which finds in p.head whether an item is its to join.  A row is a warp's, or
// several warps' where there are fewer rows than warps: each takes every so many-th part, and
// their sums are added in order.  What it costs is the wait for the kernel before it and two
// loads one after the other, the head and then everything else at a time.
template <int D, int NT, bool BF16>
__global__ void __launch_bounds__(256) kv4_join_kernel(const __grid_constant__ RowsParams p) {
    constexpr int R = 8 * NT, W = 8;
    constexpr int V = D / 32;  // values of a lane
    __shared__ float so[W][D], sl[W];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int cta = blockIdx.x;
    const int4 h = p.head[cta];
    const int parts = h.w;
    // (A workspace that calls share at the same time can hold anything; what is no item's is left alone.)
    if (parts <= 0 || cta == 0 || parts > (int)gridDim.x - cta + 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int share = ((h.z & 255) + kJoinSplit - 1) / kJoinSplit, first = blockIdx.y * share;
    const int nrows = min(share, (h.z & 255) - first), kh = h.z >> 8;
    if (nrows <= 0 || nrows > R || (unsigned)kh >= (unsigned)p.c.heads || h.x < 0 || (unsigned)h.y > (unsigned)INT32_MAX - R) return;
    const int log2 = nrows > 4 ? 0 : (nrows > 2 ? 1 : (nrows > 1 ? 2 : 3));  // warps of a row
    for (int n0 = 0; n0 < nrows; n0 += W >> log2) {
        const int n = first + n0 + (warp >> log2);
        float top = kNone, sum = 0.0f, y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = 0.0f;
        if (n < first + nrows) {
            // part 0 lies in the CTA before, as the one it began; the others continue it
            auto part = [&](int i) { return p.part + ((int64_t)(cta - 1 + i) * 2 + (i == 0 ? 1 : 0)) * (R * (D + 2)); };
            for (int i = lane; i < parts; i += 32) top = fmaxf(top, part(i)[R * D + 2 * n]);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
#pragma unroll 8
            for (int i = warp & ((1 << log2) - 1); i < parts; i += 1 << log2) {
                const float *const x = part(i);
                const float2 ml = *reinterpret_cast<const float2 *>(x + R * D + 2 * n);
                const float f = ex2(ml.x - top);
                sum = fmaf(f, ml.y, sum);
                float v[V];
                if constexpr (V == 2) {
                    const float2 u = *reinterpret_cast<const float2 *>(x + n * D + 2 * lane);
                    v[0] = u.x, v[1] = u.y;
                } else {
#pragma unroll
                    for (int e = 0; e < V; e += 4) {
                        const float4 u = *reinterpret_cast<const float4 *>(x + n * D + V * lane + e);
                        v[e] = u.x, v[e + 1] = u.y, v[e + 2] = u.z, v[e + 3] = u.w;
                    }
                }
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] = fmaf(f, v[e], y[e]);
            }
        }
        if (log2 > 0) {
#pragma unroll
            for (int e = 0; e < V; ++e) so[warp][V * lane + e] = y[e];
            if (lane == 0) sl[warp] = sum;
            __syncthreads();
            for (int w = 1; w < 1 << log2; ++w) {
                const int from = min(W - 1, warp + w);
                sum += sl[from];
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] += so[from][V * lane + e];
            }
        }
        if (n >= first + nrows || (warp & ((1 << log2) - 1)) != 0) continue;  // with several warps to a row this round is the only one
        const int r = h.y + n, tok = r / p.group;
        if ((int64_t)h.x + tok >= p.T) continue;
        const int64_t at = ((int64_t)h.x + tok) * p.q_heads + kh * p.group + (r - tok * p.group);
        const float inv = sum == 0.0f ? 0.0f : kSumUnit / sum;
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const int64_t d = at * D + V * lane + e;
            if constexpr (BF16) *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(p.out) + d) = h2_bf16(y[e] * inv, y[e + 1] * inv);
            else *reinterpret_cast<float2 *>(reinterpret_cast<float *>(p.out) + d) = make_float2(y[e] * inv, y[e + 1] * inv);
        }
        if (p.lse && lane == 0) p.lse[at] = sum == 0.0f ? -CUDART_INF_F : (top + log2f(sum)) * kLn2;
    }
}

template <typename... P, typename... A>
cudaError_t launch_one(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Dynamic shared memory above 48 KB has to be allowed once per kernel and device.
cudaError_t allow_smem(const void *kernel, int bytes, bool (&done)[kMaxDevices]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < kMaxDevices) done[dev] = true;
    return e;
}

template <int D, int NT, bool BF16>
cudaError_t launch_rows(RowsParams p, int64_t T, void *ws, cudaStream_t s) {
    constexpr size_t smem = kRowsSmem<D, NT, BF16>;
    static bool allowed[kMaxDevices] = {};
    const cudaError_t e = allow_smem((const void *)kv4_rows_kernel<D, NT, BF16>, (int)smem, allowed);
    if (e != cudaSuccess) return e;
    const int slots = sm_count() * kResident<D, NT, BF16>;
    const int grid = slots;
    p.head = static_cast<int4 *>(ws);
    p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + (size_t)grid * sizeof(int4));
    const cudaError_t r = launch_one(kv4_rows_kernel<D, NT, BF16>, grid, 32 * kWarps, smem, s, p);
    if (r != cudaSuccess || p.whole) return r;
    return launch_one(kv4_join_kernel<D, NT, BF16>, dim3(grid, kJoinSplit), 256, 0, s, p);
}

}  // namespace

size_t kv4_attention_workspace(int64_t T, int q_heads, int heads, int dim, int batch) {
    // the largest of the kernels' (fp32 has no more CTAs than bf16): a slot and two parts of 8 NT rows to a CTA
    auto need = [&](int resident, int nt) {
        return (size_t)sm_count() * resident * (sizeof(int4) + 2 * 8 * nt * (size_t)(dim + 2) * 4);
    };
    const size_t one = dim == 64 ? need(kResident<64, 1, true>, 1) : (dim == 128 ? need(kResident<128, 1, true>, 1) : need(kResident<256, 1, true>, 1));
    const size_t two = dim == 64 ? need(kResident<64, 2, true>, 2) : (dim == 128 ? need(kResident<128, 2, true>, 2) : 0);
    // the kernels run one after the other in the same memory
    const int64_t rows = T * (q_heads / heads);
    const size_t tiles = dim <= 128 && rows >= kTilesFrom ? kv4_tiles_workspace(T, q_heads / heads, heads, dim, batch, kTilesFrom) : 0;
    size_t most = one > two ? one : two;
    const size_t chunk = rows >= kTilesFrom ? kv4_chunk_workspace(T, q_heads / heads, heads, dim, batch, kTilesFrom) : 0;
    most = most > tiles ? most : tiles;
    most = most > chunk ? most : chunk;
    return (most + 255) & ~(size_t)255;
}

cudaError_t launch_kv4_attention(const void *q, bool bf16, int64_t T, int q_heads, int64_t qts, int64_t qhs,
                                 const Kv4Cache &c, const Kv4Batch &bt, float scale, bool causal, int64_t window,
                                 int64_t max_q, void *out, float *lse, void *ws, cudaStream_t s) {
    RowsParams p = {};
    p.q = q, p.qts = qts, p.qhs = qhs, p.q_heads = q_heads, p.group = q_heads / c.heads, p.T = T;
    p.c = c, p.bt = bt, p.scale = scale, p.causal = causal;
    p.window = window > 0 && window < INT32_MAX ? (int)window : INT32_MAX;
    // Longer runs of rows go to the kernels that unpack a code for 128 rows or more at a time.  max_q is a hint: without
    // them every sequence is this one's.
    const int64_t rows = (max_q > 0 && max_q < T ? max_q : T) * p.group;
    const bool tiles = rows >= kTilesFrom;
    // One sequence is theirs whatever it has of the rows, and this kernel is not launched for the rest: a prompt of 130
    // tokens takes 17 us instead of 21.  (One with a few of T's rows is slower there, and still right; max_q tells.)
    const int rows_min = bt.batch == 1 ? 1 : kTilesFrom;
    p.rows_max = tiles ? rows_min - 1 : INT32_MAX;
    p.out = out, p.lse = lse, p.status = device_status_ptr();
    const bool many = 2 * (int64_t)bt.batch * c.heads >= sm_count();
    const int64_t span = (int64_t)p.window + 16 / p.group + 2, held = (int64_t)bt.max_pages << c.page_log2;  // as in seq_of()
    p.whole = (held < span ? held : span) <= (many ? 2 : 1) * kWholeTiles * kTile;
    p.magic[0] = 0x64086408u, p.magic[1] = 0x64806480u;
    if (tiles) {
        const cudaError_t e = bf16 && c.dim <= 128
                                  ? launch_kv4_tiles(q, T, q_heads, qts, qhs, c, bt, scale, causal, p.window, rows_min, out, lse, ws, s)
                                  : launch_kv4_chunks(q, bf16, T, q_heads, qts, qhs, c, bt, scale, causal, p.window, rows_min, out, lse, ws, s);
        if (e != cudaSuccess || rows_min == 1) return e;
    }
    const bool two = rows > 8;
    if (c.dim == 64) {
        if (two) return bf16 ? launch_rows<64, 2, true>(p, T, ws, s) : launch_rows<64, 2, false>(p, T, ws, s);
        return bf16 ? launch_rows<64, 1, true>(p, T, ws, s) : launch_rows<64, 1, false>(p, T, ws, s);
    }
    if (c.dim == 128) {
        if (two) return bf16 ? launch_rows<128, 2, true>(p, T, ws, s) : launch_rows<128, 2, false>(p, T, ws, s);
        return bf16 ? launch_rows<128, 1, true>(p, T, ws, s) : launch_rows<128, 1, false>(p, T, ws, s);
    }
    return bf16 ? launch_rows<256, 1, true>(p, T, ws, s) : launch_rows<256, 1, false>(p, T, ws, s);
}

}  // namespace bitnet
