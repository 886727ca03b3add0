// decode.cu -- attention of one new token per request over the paged key-value cache
// (include/inkling_paged_attn.h, inkling_rel_attn_decode) and its C entry point.
//
// For request n, KV head g and the query heads h of its group:
//   z_j = scale <q_h, k_j> + (d < R ? profiles[n, h, d] : 0),  d = len - 1 - j
//   m = max z_j, l = sum exp(z_j - m), O = sum exp(z_j - m) v_j
//   lse = log(exp(sink) + exp(m) l), out = O exp(m - lse)
// in one pass over the keys with the running maximum and sum of the softmax; parts of the
// keys are joined by their (m, l, O).
//
// Every cached value is read once and used for the Hq / Hkv query heads of its group, 2 to
// 16 products per byte: bound by HBM. So the work is laid out for bytes in flight:
//   * each warp is a worker of its own, eight to an SM whatever the batch. The tiles of KT
//     keys of all (request, KV head) units are numbered through and each worker takes an
//     equal run of them, so ragged batches and single long requests load every SM the same.
//     The run is found on the device from the lengths: nothing about them is needed on the
//     host. A unit that is cut leaves its parts in the workspace and a second kernel joins
//     them in the order of the keys.
//   * a worker streams its tiles through a private cp.async ring in shared memory that
//     runs on over the ends of units (the next unit's tiles are on their way while the last
//     one's result is written) with no block barrier anywhere in the loop. cp.async with
//     one row address per key takes any page size and any strides, and fills the rows of
//     keys that are not allowed with zeros, so nothing that stands in such a place (NaN,
//     infinities) reaches a product. The profile entries of a tile's distances come through
//     the same ring.
//   * products are mma.sync m16n8k16: with a group of 8 heads or fewer a tile is far too
//     narrow for tcgen05 (64 or 128 rows of M), and the tensor pipe is idle most of the
//     time anyway. S[heads, keys] = Q K^T puts the heads in M, so its accumulators are
//     already the B operand of O^T[d, heads] = V^T P^T: no shuffle between the products.
//     K fragments come by ldmatrix, V fragments by its transposing form.
//   * probabilities enter the second product as a sum of 16-bit numbers (p, what its
//     rounding left, and for BF16 what that one's left), which costs one or two more mma on
//     an idle pipe and keeps the FP32 result to 2^-22 of a probability or less, where one
//     BF16 number would keep 2^-8. Each tile's product starts from zero and is added to O in
//     FP32, as the tensor pipe's own sum is cut off, not rounded, and would drift.
// e4m3 caches: a code is exact in FP16, so both products run in FP16 with FP32 sums; the
// scales stay outside the products. q (BF16) is first multiplied by a power of two per
// head that brings its largest value into [1, 2): exact but for values below 2^-14 of
// the largest, whose error (2^-25 of it) is under the FP32 sum's own.
//
// Measured (GPU time of a call, of the measured copy bandwidth): eight requests of 32767
// tokens, 32 / 8 heads of 128, profiles of 4096: 176 us, 6.12 TB/s, 0.93; one of 32768: 30.7
// us, 4.38 TB/s, 0.67 (of it 5 us until the first tile is in and 4 us for the join); 64
// requests of 16 to 4096 tokens: 41.3 us, 4.79 TB/s, 0.73; 24 requests of 8191 to 32768
// tokens in e4m3, 32 / 4 heads: 87.2 us, 5.28 TB/s, 0.81 (a tile's dependent instructions
// take about 2,600 cycles for its 8 KB with two warps to a scheduler, which is what HBM
// takes as well; calls of 92 to 95 us were seen on other boards). A plain sum over as many
// bytes takes 181, 29.0, 38.3 and 89.4 us.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace {

using namespace ira;

constexpr int kWarps = 4;
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 320;
constexpr int kMaxWorkers = kMaxCtas * kWarps;  // workspace slots: two per worker
// One CTA per unit, with no split, up to these sizes: tiles of each of its warps, and units
// of the call. Both sides, GPU us whole (its warps) and split, with 16 / 4 heads of 128 (4 units
// to a request) and requests of 1 to 2048 tokens, W the window:
//   requests  BF16, W 512     BF16, W 1024    e4m3, W 512     e4m3, W 1024
//     1       6.9 (8) 10.7    10.7 (8)  9.5    5.7 (8) 10.0    8.7 (8) 11.6
//     4       7.2 (8) 10.9    10.9 (8) 10.9    5.9 (8)  9.8    8.9 (8) 11.5
//    16       7.6 (8) 11.9    10.8 (8) 11.6    6.1 (8) 10.6    8.8 (8) 11.9
//    32       7.8 (8) 12.2    12.3 (8) 12.3    6.1 (8) 11.9    9.0 (8) 12.4
//    64      11.8 (4) 13.9    15.8 (8) 15.3    8.9 (4) 11.4   13.6 (4) 12.9
//   128      17.2 (4) 17.7    22.4 (8) 20.1   12.6 (4) 13.6   17.6 (4) 15.6
//   200      23.3 (4) 21.0    34.4 (8) 24.5   18.5 (4) 17.2   24.7 (4) 20.1
// So the rule is right but for two corners, where the split would be 1.2 us (a lone request with
// 33 to 64 tiles of 16 keys) and 0.7 to 2 us (129 to 512 units of 17 to 32 tiles of 32) faster.
constexpr int kWholeTiles = 8;
constexpr int kWholeUnits = 512;
constexpr int kJoinThreads = 256;
constexpr int kJoinBatch = 6;                   // parts that a lane of it loads at once

// A worker's last unit, if it began there and did not end: first row of out, rows, and how
// many of the next workers have the unit's other parts (their first ones).
struct alignas(16) Rec {
    long long row;
    int heads, more;
};

struct DecodeParams {
    int N, Hq, Hkv, group, hblocks, unit_heads, R, W, M, num_pages, cap;
    PageDivisor page;
    int64_t page_stride, token_stride, head_stride;  // bytes
    float scale_log2;
    const uint16_t* q;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const float* k_scale;
    const float* v_scale;
    const uint16_t* profiles;
    const float* sink;
    const int32_t* table;
    const int32_t* lens;
    float* out;
    float* lse;
    Rec* rec;          // [workers of the grid]
    float2* part_ml;   // [2 * workers][unit_heads]
    float* part_o;     // [2 * workers][unit_heads][D]
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// c += a b, 16 x 8 x 16, FP32 sums of BF16 or FP16 products
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// four e4m3 codes as two FP16 pairs, exactly
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_bf16x2(lo, hi);
    }
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
}

// Shape of one instantiation. D head_dim, NT groups of 8 query heads (1 or 2), F8 e4m3
// cache. A tile is 8 KB of K and V in every form but the smallest, so that the two or three
// of each worker that are on their way are 128 KB or more on an SM.
template <int D_, int NT_, bool F8_>
struct Shape {
    static constexpr int D = D_, NT = NT_;
    static constexpr bool F8 = F8_;
    static constexpr int ES = F8 ? 1 : 2;
    static constexpr int RB = D * ES;                       // bytes of a row
    static constexpr int CPR = RB / 16;                     // 16-byte chunks of a row
    static constexpr int KT = (D == 128 && !F8) ? 16 : 32;  // keys of a tile
    // e4m3: probabilities are taken 2^7 times, as FP16 has no exponent below 2^-24: so each of
    // them is off by 2^-32 of the largest at most (they stay below 2^15, as the running
    // maximum lags by 2^8 at most), and long tails of small ones are not lost.
    static constexpr float LIFT = F8 ? 7.f : 0.f;
    static_assert(kRescaleThreshold + LIFT <= 15.f, "FP16 ends below 2^16");
    static constexpr int STAGES = 3;
    static constexpr int SIDE = KT * RB;                    // bytes of K (or V) in a stage
    static constexpr int BCH = KT / 8 + 1;                  // 16-byte chunks that hold KT profile entries
    static constexpr int STAGE = 2 * SIDE + 8 * NT * BCH * 16;
    // Tiles (and unit starts) that a worker takes at least. A part is written and read again,
    // 1 KB for each head: no more parts than their traffic stays around half of the tiles'.
    // Measured with one request (GPU time): 4096 tokens, 8 x 4 heads 11.6 us with 2 and
    // 13.1 us with 4; 32768 tokens, 1 x 16 heads 22.1 us with 2 and 18.5 us with 4.
    static constexpr int MIN_TILES = 2 * NT;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int OROW = D + 4;                      // floats of a head's row when warps join (no bank conflicts)
    static_assert(8 * NT * OROW * 4 <= RING, "the rings hold the warps' results when they join");
    // chunk c of row r stands at chunk c ^ swz(r): ldmatrix's eight rows use all banks
    __device__ static __forceinline__ int swz(int row) { return RB >= 128 ? (row & 7) : ((row >> 1) & 3); }
};

struct Span {  // allowed keys [lo, len) of a request and its tiles (at least one)
    int lo, len, tiles;
};
template <int KT>
__device__ __forceinline__ Span span_of(const DecodeParams& p, int raw_len) {
    Span s;
    s.len = min(max(raw_len, 0), p.cap);
    s.lo = p.W > 0 ? max(s.len - p.W, 0) : 0;
    s.tiles = max((s.len - s.lo + KT - 1) / KT, 1);
    return s;
}

// lse of a row from the maximum of its keys' logits, that of those and the sink (log2 units),
// and the sum over both relative to it; the sink itself where no key is left.
__device__ __forceinline__ float lse_of(float keys, float top, float total, const float* sink, int64_t at) {
    if (keys == -INFINITY && total <= 1.f) return sink ? sink[at] : -INFINITY;
    return (top + log2f(total)) * kLn2;
}

// exp2(x - top), 1 where both are the same infinity
__device__ __forceinline__ float weight(float x, float top) { return x == top ? 1.f : ex2_approx(x - top); }

enum : int { kFirst = 1, kLast = 2, kBegins = 4, kEnds = 8 };  // of a run of tiles of one unit

// Position in the numbered tiles: request, unit of it (KV head and block of query heads),
// tile of that; `at` counts tiles and unit starts from the worker's first one.
struct Cursor {
    Span s;
    int n, kvh, hb, t, next_len, at;
};

// WHOLE (4 or 8 warps): a CTA for each unit and no split. Its warps take the unit's tiles in
// turn and join through shared memory: no prefix sums at the start, no second kernel at the
// end. WHOLE == 0: the grid's warps are workers with an even share each of all tiles. A unit counts
// one more than its tiles there, which is about what loading its query and writing its
// result take, so that runs of short requests are not the last to finish.
template <class S, int WHOLE>
__global__ void __launch_bounds__(32 * (WHOLE ? WHOLE : kWarps), WHOLE == 8 ? 1 : kCtasPerSm)
    decode_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int WARPS = WHOLE ? WHOLE : kWarps, THREADS = 32 * WARPS;
    constexpr int D = S::D, NT = S::NT, KT = S::KT, ST = S::STAGES;
    constexpr bool F8 = S::F8;
    constexpr int NS = KT / 8;  // S accumulator tiles of 8 keys
    constexpr int STEP = WHOLE ? WARPS : 1;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int4 s_tile[WARPS][ST];  // allowed keys, kFirst .., distance of the last key (dlo), Cursor::at
    __shared__ int4 s_run[WARPS][ST];   // of a run's first tile: request, KV head, first query head, length
    __shared__ long long s_sum[WARPS];
    __shared__ long long s_base[WARPS];
    __shared__ int s_n[WARPS], s_len[WARPS];
    __shared__ float2 s_ml[WARPS][8 * NT];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int units = p.Hkv * p.hblocks;  // per request
    const uint32_t ring = smem_u32(smem) + warp * S::RING;

    release_successor();
    wait_for_predecessor();
    Cursor cur{};
    // worker w has share tiles (and unit starts), the first `longer` workers one more
    long long all = 0, first = 0, share = 0;
    int limit = 0, worker = 0, workers = 0, longer = 0;
    auto begin_of = [&](int w) { return w * share + min(w, longer); };
    if constexpr (WHOLE) {
        cur.n = blockIdx.x / units;
        cur.kvh = (blockIdx.x - cur.n * units) / p.hblocks;
        cur.hb = blockIdx.x - cur.n * units - cur.kvh * p.hblocks;
        cur.t = warp;
        cur.s = span_of<KT>(p, p.lens[cur.n]);
    } else {
        const int chunk = (p.N + THREADS - 1) / THREADS;
        const int n0 = min(tid * chunk, p.N), n1 = min(n0 + chunk, p.N);
        long long own = 0;
        for (int n = n0; n < n1; ++n) own += span_of<KT>(p, p.lens[n]).tiles + 1;
        long long inc = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += x;
        }
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        long long before = inc - own;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) before += s_sum[w];
            all += s_sum[w];
        }
        all *= units;
        before *= units;
        const long long enough = max(all / S::MIN_TILES, 1ll);
        workers = int(enough < (long long)gridDim.x * WARPS ? enough : (long long)gridDim.x * WARPS);
        share = all <= 0x7fffffff ? uint32_t(all) / uint32_t(workers) : all / workers;
        longer = int(all - share * workers);
        // neighbours in the order of the tiles are on different SMs
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const long long from = begin_of(w * gridDim.x + blockIdx.x);
            if (before <= from && from < before + own * units) {
                long long at = before;
                int n = n0, len;
                for (;; ++n) {
                    len = p.lens[n];
                    const long long size = (long long)(span_of<KT>(p, len).tiles + 1) * units;
                    if (from < at + size) break;
                    at += size;
                }
                s_n[w] = n;
                s_len[w] = len;
                s_base[w] = at;
            }
        }
        __syncthreads();
        worker = warp * gridDim.x + blockIdx.x;
        if (worker >= workers) {
            if (lane == 0) p.rec[worker] = Rec{0, 0, 0};
            return;
        }
        first = begin_of(worker);
        limit = int(share) + (worker < longer ? 1 : 0);
        cur.n = s_n[warp];
        cur.next_len = cur.n + 1 < p.N ? p.lens[cur.n + 1] : 0;
        cur.s = span_of<KT>(p, s_len[warp]);
        const long long local = first - s_base[warp];
        const int u = all <= 0x7fffffff ? int(uint32_t(local) / uint32_t(cur.s.tiles + 1)) : int(local / (cur.s.tiles + 1));
        cur.kvh = u / p.hblocks;
        cur.hb = u - cur.kvh * p.hblocks;
        cur.t = int(local - (long long)u * (cur.s.tiles + 1)) - 1;
        if (cur.t < 0) cur.t = 0, cur.at = 1;  // the range begins with the unit's start
    }

    // ---- producer: lane r < KT looks key r of a tile up, all lanes copy
    constexpr uint32_t kAll = KT == 32 ? 0xffffffffu : (1u << (KT & 31)) - 1u;
    const int my_key = lane & (KT - 1);
    auto there = [&](const Cursor& c) { return WHOLE ? c.t < c.s.tiles : c.at < limit; };
    auto advance = [&](Cursor& c) {
        c.t += STEP;
        if constexpr (!WHOLE) {
            ++c.at;
            if (c.t < c.s.tiles) return;
            c.t = 0;
            ++c.at;
            if (++c.hb < p.hblocks) return;
            c.hb = 0;
            if (++c.kvh < p.Hkv) return;
            c.kvh = 0;
            ++c.n;
            c.s = span_of<KT>(p, c.next_len);
            c.next_len = c.n + 1 < p.N ? p.lens[c.n + 1] : 0;
        }
    };
    auto lookup = [&](const Cursor& c) {  // -1: not allowed
        const int j = c.s.lo + c.t * KT + my_key;
        return j < c.s.len ? p.table[int64_t(c.n) * p.M + p.page.index(j)] : -1;
    };
    // Issues a tile's copies. It stands between the products of every tile, so it is kept to few
    // instructions: no division, and one or two page bases where a tile meets no third page.
    auto issue = [&](const Cursor& c, int i, int stage, int page) {
        const int j0 = c.s.lo + c.t * KT;
        const int head0 = c.kvh * p.group + c.hb * 8 * NT;
        const bool ok = page >= 0 && page < p.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & kAll;
        const bool run = i == 0 || (!WHOLE && c.t == 0), ends = c.t == c.s.tiles - 1;
        const int dlo = c.s.len - KT - j0;  // distance of the tile's last key
        if (lane == 0) {
            s_tile[warp][stage] = make_int4(int(mask),
                                            (run ? kFirst : 0) | (ends || c.at + 1 >= limit ? kLast : 0) |
                                                (c.t == 0 ? kBegins : 0) | (ends ? kEnds : 0),
                                            dlo, c.at);
            if (run) s_run[warp][stage] = make_int4(c.n, c.kvh, head0, c.s.len);
        }
        const uint32_t dst = ring + stage * S::STAGE;
        constexpr int ROWS = 32 / S::CPR;  // of a copy of 16 bytes per lane
        const int r0 = lane / S::CPR, ch = lane % S::CPR;
        const int64_t head = c.kvh * p.head_stride + ch * 16;
        const int offset = j0 - p.page.index(j0) * p.page.size;  // of the first key in its page
        const int split = p.page.size - offset;                  // keys up to that page's end
        if (p.page.size >= KT) {
            const int pa = __shfl_sync(0xffffffffu, page, 0), pb = __shfl_sync(0xffffffffu, page, min(split, KT - 1));
            int64_t a = pa * p.page_stride + (offset + r0) * p.token_stride + head;
            // The usual tile: every key allowed, all in one page. Where rows of a head follow each
            // other ([pages, heads, page_size, D]) the copies differ by constants alone, which takes
            // 8-bit caches 2 % less time.
            if (mask == kAll && split >= KT && p.token_stride == S::RB) {
                const uint8_t *k = p.k_cache + a, *v = p.v_cache + a;
#pragma unroll
                for (int x = 0; x < KT / ROWS; ++x) {
                    const int r = x * ROWS + r0;
                    const uint32_t to = dst + r * S::RB + ((ch ^ S::swz(r)) << 4);
                    cp_async_16(to, k + x * ROWS * S::RB, 16u);
                    cp_async_16(to + S::SIDE, v + x * ROWS * S::RB, 16u);
                }
            } else if (mask == kAll && split >= KT) {
                const uint8_t *k = p.k_cache + a, *v = p.v_cache + a;
#pragma unroll
                for (int x = 0; x < KT / ROWS; ++x) {
                    const int r = x * ROWS + r0;
                    const uint32_t to = dst + r * S::RB + ((ch ^ S::swz(r)) << 4);
                    cp_async_16(to, k, 16u);
                    cp_async_16(to + S::SIDE, v, 16u);
                    k += ROWS * p.token_stride;
                    v += ROWS * p.token_stride;
                }
            } else {
                int64_t b = pb * p.page_stride + (r0 - split) * p.token_stride + head;
#pragma unroll
                for (int x = 0; x < KT / ROWS; ++x) {
                    const int r = x * ROWS + r0;
                    const bool in = (mask >> r) & 1u;
                    const int64_t off = in ? (r < split ? a : b) : 0;
                    const uint32_t to = dst + r * S::RB + ((ch ^ S::swz(r)) << 4);
                    cp_async_16(to, p.k_cache + off, in ? 16u : 0u);
                    cp_async_16(to + S::SIDE, p.v_cache + off, in ? 16u : 0u);
                    a += ROWS * p.token_stride;
                    b += ROWS * p.token_stride;
                }
            }
        } else {  // pages shorter than a tile: each key's row by itself
            const int j = j0 + my_key;
            const int64_t at =
                ok ? page * p.page_stride + (j - p.page.index(j) * p.page.size) * p.token_stride : 0;
#pragma unroll
            for (int x = 0; x < KT / ROWS; ++x) {
                const int r = x * ROWS + r0;
                const bool in = (mask >> r) & 1u;
                const int64_t row = __shfl_sync(0xffffffffu, at, r);
                const int64_t off = in ? row + head : 0;
                const uint32_t to = dst + r * S::RB + ((ch ^ S::swz(r)) << 4);
                cp_async_16(to, p.k_cache + off, in ? 16u : 0u);
                cp_async_16(to + S::SIDE, p.v_cache + off, in ? 16u : 0u);
            }
        }
        // profile entries of the distances [dlo, dlo + KT), in whole chunks of 8
        const int heads = min(8 * NT, p.group - c.hb * 8 * NT);
        if (p.R > 0 && dlo < p.R) {
            const int c0 = dlo >> 3;
            const uint16_t* const first_row = p.profiles + (int64_t(c.n) * p.Hq + head0) * p.R;
#pragma unroll
            for (int x = lane; x < 8 * NT * S::BCH; x += 32) {
                const int h = x / S::BCH, ch = c0 + x - h * S::BCH;
                const bool in = h < heads && ch >= 0 && ch < (p.R >> 3);
                const int64_t off = in ? int64_t(h) * p.R + ch * 8 : 0;
                cp_async_16(dst + 2 * S::SIDE + x * 16, first_row + off, in ? 16u : 0u);
            }
        }
        if (!WHOLE && run) {  // q and the sink are loaded when the tile's turn comes: warm L2 for that
            if (lane < heads * D / 64) prefetch_l2(p.q + (int64_t(c.n) * p.Hq + head0) * D + lane * 64);
            if (lane == 31 && p.sink) prefetch_l2(p.sink + int64_t(c.n) * p.Hq + head0);
        }
    };

    // ---- query of a unit: fragments (BF16 pairs as they stand in memory) and the sink
    struct Query {
        uint32_t a[D / 16][2 * NT];
        float sink[NT];
    };
    int heads = 0;  // query heads of the unit
    auto first_head = [&](const Cursor& c) { return c.kvh * p.group + c.hb * 8 * NT; };
    auto heads_from = [&](int kvh, int from) { return min(8 * NT, (kvh + 1) * p.group - from); };
    auto load_query = [&](Query& q, int n, int from, int count) {
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            const int h = g + 8 * r;
            const int64_t at = int64_t(n) * p.Hq + from + h;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + at * D);
            q.sink[r] = p.sink && h < count ? p.sink[at] : -INFINITY;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                // BF16: columns 16 ks + {2t, 2t+1} and + 8; e4m3: 16 ks + {4t .. 4t+3}, the
                // order in which a code word holds them (K uses the same one)
                const int w0 = F8 ? 8 * ks + 2 * t : 8 * ks + t, w1 = F8 ? w0 + 1 : w0 + 4;
                q.a[ks][2 * r] = h < count ? src[w0] : 0u;
                q.a[ks][2 * r + 1] = h < count ? src[w1] : 0u;
            }
        }
    };

    Query qa;
    float zscale[NT];
    float o[D / 16][NT][4];
    float mx[NT], sum[NT];
    auto start = [&](int kvh) {  // of a unit, its query in qa
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            zscale[r] = p.scale_log2;
            qa.sink[r] *= kLog2e;
            mx[r] = -INFINITY;
            sum[r] = 0.f;
            if constexpr (F8) {
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 x = unpack2<false>(qa.a[ks][2 * r + e]);
                        top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^e <= top < 2^(e+1) (zero, subnormal and infinite rows: the nearest normal power)
                const int e = min(max(int(__float_as_uint(top) >> 23) - 127, -126), 126);
                const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float2 x = unpack2<false>(qa.a[ks][2 * r + y]);
                        qa.a[ks][2 * r + y] = pack2<true>(x.x * down, x.y * down);
                    }
                zscale[r] *= __uint_as_float(uint32_t(127 + e) << 23) * p.k_scale[kvh];
                if (zscale[r] == 0.f) zscale[r] = 0x1p-126f;  // masked entries are -inf times this
            }
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[m][r][e] = 0.f;
        }
    };

    if constexpr (WHOLE) {
        heads = heads_from(cur.kvh, first_head(cur));
        load_query(qa, cur.n, first_head(cur), heads);
    }
    int page = -1, made = 0;
    {
        // the first lookups go out together
        Cursor at[ST];
        int pages[ST];
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            at[i] = cur;
            if (i > 0) {
                at[i] = at[i - 1];
                if (there(at[i - 1])) advance(at[i]);
            }
            pages[i] = there(at[i]) ? lookup(at[i]) : -1;
        }
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) {
            if (there(at[i])) issue(at[i], made++, i, pages[i]);
            cp_async_commit();
        }
        cur = at[ST - 1];
        page = pages[ST - 1];
    }
    if constexpr (WHOLE) start(cur.kvh);

    [[maybe_unused]] Query qn;  // the next unit's query, where registers allow
    [[maybe_unused]] bool begins = false;
    [[maybe_unused]] int4 run = make_int4(0, 0, 0, 0);
    Rec rec{0, 0, 0};

    int stage = 0;
    for (int i = 0; i < made; ++i) {
        cp_async_wait_group<ST - 2>();
        __syncwarp();  // the tile is in, and every lane is done with the previous one's stage
        const int behind = stage == 0 ? ST - 1 : stage - 1, ahead = stage == ST - 1 ? 0 : stage + 1;
        const bool had_next = i + 1 < made;
        const int4 tile = s_tile[warp][stage];
        const uint32_t mask = uint32_t(tile.x);
        const int flags = tile.y, dlo = tile.z;
        const uint32_t kbase = ring + stage * S::STAGE, vbase = kbase + S::SIDE, bbase = vbase + S::SIDE;

        if constexpr (!WHOLE) {
            if (flags & kFirst) {
                begins = flags & kBegins;
                run = s_run[warp][stage];
                heads = heads_from(run.y, run.z);
                if (NT == 1 && i > 0) qa = qn;
                else load_query(qa, run.x, run.z, heads);
                start(run.y);
            }
            // one group of heads leaves the registers to have the next unit's query on its way
            if (NT == 1 && had_next && (s_tile[warp][ahead].y & kFirst)) {
                const int4 next = s_run[warp][ahead];
                load_query(qn, next.x, next.z, heads_from(next.y, next.z));
            }
        }
        stage = ahead;

        // The next tile's copies are issued behind the first product, whose latency they hide in.
        auto produce = [&] {
            if (there(cur)) {
                issue(cur, made++, behind, page);
                advance(cur);
                if (there(cur)) page = lookup(cur);
            }
            cp_async_commit();
        };
        if (mask == 0) {
            produce();
        } else {
            // lane's row and chunk parity in the 16-key ldmatrix of either side
            const int lrow = (lane & 7) + ((lane >> 4) << 3), lch = (lane >> 3) & 1;
            const int lswz = S::swz(lane & 7);

            // ---- S = Q K^T
            float s[NS][4];
#pragma unroll
            for (int x = 0; x < NS; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[x][e] = 0.f;
#pragma unroll
            for (int c = 0; c < S::CPR / 2; ++c) {  // pairs of 16-byte chunks
#pragma unroll
                for (int kk = 0; kk < KT / 16; ++kk) {
                    uint32_t f[4];
                    ldmatrix_x4(kbase + (kk * 16 + lrow) * S::RB + (((2 * c + lch) ^ lswz) << 4), f);
                    if constexpr (!F8) {
                        const uint32_t a1 = NT == 2 ? qa.a[c][2 * (NT - 1)] : 0u, a3 = NT == 2 ? qa.a[c][2 * NT - 1] : 0u;
                        mma16816<false>(s[2 * kk], qa.a[c][0], a1, qa.a[c][1], a3, f[0], f[1]);
                        mma16816<false>(s[2 * kk + 1], qa.a[c][0], a1, qa.a[c][1], a3, f[2], f[3]);
                    } else {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {  // the pair's two chunks: 16 columns each
                            const uint32_t* a = qa.a[2 * c + x];
                            const uint32_t a1 = NT == 2 ? a[2 * (NT - 1)] : 0u, a3 = NT == 2 ? a[2 * NT - 1] : 0u;
                            uint32_t b0, b1, b2, b3;
                            e4m3x4_to_f16x4(f[x], b0, b1);
                            e4m3x4_to_f16x4(f[x + 2], b2, b3);
                            mma16816<true>(s[2 * kk], a[0], a1, a[1], a3, b0, b1);
                            mma16816<true>(s[2 * kk + 1], a[0], a1, a[1], a3, b2, b3);
                        }
                    }
                }
            }
            produce();

            // ---- logits in log2 units are s zs; with profile entries they are made here
            float zs[NT];
#pragma unroll
            for (int r = 0; r < NT; ++r) zs[r] = zscale[r];
            if (p.R > 0 && dlo < p.R) {
#pragma unroll
                for (int r = 0; r < NT; ++r) {
                    // entry of key x of the tile: the one of distance dlo + KT - 1 - x
                    const uint32_t at = bbase + (g + 8 * r) * (S::BCH * 16) + ((dlo & 7) + KT - 1 - 2 * t) * 2;
#pragma unroll
                    for (int x = 0; x < NS; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            s[x][2 * r + e] = fmaf(__uint_as_float(lds_u16(at - (8 * x + e) * 2) << 16), kLog2e,
                                                   s[x][2 * r + e] * zs[r]);
                    zs[r] = 1.f;
                }
            }
            if (mask != kAll) {
#pragma unroll
                for (int r = 0; r < NT; ++r)
#pragma unroll
                    for (int x = 0; x < NS; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!((mask >> (8 * x + 2 * t + e)) & 1u)) s[x][2 * r + e] = -INFINITY;
            }
            // ---- the running maximum moves only when a logit passes it by 2^8, which each lane
            // sees for its own entries: no exchange in the usual tile. Compared as the exponents
            // are taken below, from the lifted maximum: at 2^24 and above that is rounded by as
            // much as 4, and a probability must still fit into FP16.
            float top[NT];
            bool grows = false;
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                top[r] = -INFINITY;
#pragma unroll
                for (int x = 0; x < NS; ++x) top[r] = fmax3(top[r], s[x][2 * r], s[x][2 * r + 1]);
                top[r] *= zs[r];
                grows |= top[r] - (mx[r] - S::LIFT) > kRescaleThreshold + S::LIFT;
            }
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int r = 0; r < NT; ++r) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                    const float now = fmaxf(mx[r], top[r]);
                    const float f = weight(mx[r], now);
                    mx[r] = now;
                    sum[r] *= f;
                    // heads of this thread's O columns: 2t, 2t + 1 (+ 8 r)
                    const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
                    for (int m = 0; m < D / 16; ++m) {
                        o[m][r][0] *= f0;
                        o[m][r][1] *= f1;
                        o[m][r][2] *= f0;
                        o[m][r][3] *= f1;
                    }
                }
            }
            constexpr int TERMS = F8 ? 2 : 3;  // 16-bit numbers of a probability
            uint32_t pr[TERMS][NT][NS];
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                const float ref = mx[r] == -INFINITY ? 0.f : mx[r] - S::LIFT;
#pragma unroll
                for (int x = 0; x < NS; ++x) {
                    float p0 = ex2_approx(fmaf(s[x][2 * r], zs[r], -ref));
                    float p1 = ex2_approx(fmaf(s[x][2 * r + 1], zs[r], -ref));
                    sum[r] += p0 + p1;
#pragma unroll
                    for (int k = 0; k < TERMS; ++k) {
                        pr[k][r][x] = pack2<F8>(p0, p1);
                        const float2 b = unpack2<F8>(pr[k][r][x]);
                        p0 -= b.x;
                        p1 -= b.y;
                    }
                }
            }

            // ---- O^T += V^T P^T
#pragma unroll
            for (int c = 0; c < S::CPR / 2; ++c) {
                constexpr int MT = F8 ? 2 : 1;  // 16-column tiles of a pair of chunks
                float acc[MT][NT][4];
#pragma unroll
                for (int x = 0; x < MT; ++x)
#pragma unroll
                    for (int r = 0; r < NT; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[x][r][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < KT / 16; ++kk) {
                    uint32_t f[4];
                    ldmatrix_x4_trans(vbase + (kk * 16 + lrow) * S::RB + (((2 * c + lch) ^ lswz) << 4), f);
#pragma unroll
                    for (int x = 0; x < MT; ++x) {
                        uint32_t a0 = f[0], a1 = f[1], a2 = f[2], a3 = f[3];
                        if constexpr (F8) {
                            // a 16-bit unit holds columns 2g, 2g + 1 of one key: regroup by column
                            e4m3x4_to_f16x4(__byte_perm(f[x], 0, 0x3120), a0, a1);
                            e4m3x4_to_f16x4(__byte_perm(f[x + 2], 0, 0x3120), a2, a3);
                        }
#pragma unroll
                        for (int r = 0; r < NT; ++r)
#pragma unroll
                            for (int k = TERMS - 1; k >= 0; --k)
                                mma16816<F8>(acc[x][r], a0, a1, a2, a3, pr[k][r][2 * kk], pr[k][r][2 * kk + 1]);
                    }
                }
#pragma unroll
                for (int x = 0; x < MT; ++x)
#pragma unroll
                    for (int r = 0; r < NT; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[MT * c + x][r][e] += acc[x][r][e];
            }
        }

        if constexpr (!WHOLE) {
            if (flags & kLast) {
                const int n = run.x, head0 = run.z;
                const bool ends = flags & kEnds, whole = begins && ends;
                const float vs = F8 ? p.v_scale[run.y] : 1.f;
                const int slot = 2 * worker + (begins ? 1 : 0);
#pragma unroll
                for (int r = 0; r < NT; ++r) {
                    const int h = g + 8 * r;
                    const float m0 = mx[r] - S::LIFT;  // what the sum and O are relative to
                    float l = sum[r];
                    l += __shfl_xor_sync(0xffffffffu, l, 1);
                    l += __shfl_xor_sync(0xffffffffu, l, 2);
                    float mul = vs;
                    if (whole) {
                        const float top = fmaxf(m0, qa.sink[r]);
                        const float f = weight(m0, top);
                        const float tot = top == -INFINITY ? 0.f : l * f + weight(qa.sink[r], top);
                        mul = tot == 0.f ? 0.f : vs * f / tot;
                        if (t == 0 && h < heads) {
                            const int64_t at = int64_t(n) * p.Hq + head0 + h;
                            p.lse[at] = lse_of(m0, top, tot, p.sink, at);
                        }
                    } else if (t == 0 && h < heads) {
                        p.part_ml[int64_t(slot) * p.unit_heads + h] = make_float2(m0, l);
                    }
                    float* const to = whole ? p.out + (int64_t(n) * p.Hq + head0 + 8 * r) * D
                                            : p.part_o + (int64_t(slot) * p.unit_heads + 8 * r) * D;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = __shfl_sync(0xffffffffu, mul, 8 * t + 4 * e);
                        const int hc = 2 * t + e;  // this thread's O columns
                        if (8 * r + hc >= heads) continue;
#pragma unroll
                        for (int m = 0; m < D / 16; ++m) {
                            if constexpr (F8) {
                                *reinterpret_cast<float2*>(to + hc * D + 16 * m + 2 * g) =
                                    make_float2(o[m][r][e] * f, o[m][r][2 + e] * f);
                            } else {
                                to[hc * D + 16 * m + g] = o[m][r][e] * f;
                                to[hc * D + 16 * m + g + 8] = o[m][r][2 + e] * f;
                            }
                        }
                    }
                }
                if (begins && !ends) {
                    // the worker of the unit's last tile, which is tiles - 1 - t behind this one
                    const Span sp = span_of<KT>(p, run.w);
                    const long long rest = sp.tiles - 1 - (run.w - KT - dlo - sp.lo) / KT;
                    const long long at = first + tile.w + rest, split = longer * (share + 1);
                    const int owner = int(at < split ? at / (share + 1) : longer + (at - split) / share);
                    rec = Rec{int64_t(n) * p.Hq + head0, heads, owner - worker};
                }
            }
        }
    }

    if constexpr (!WHOLE) {
        if (lane == 0) p.rec[worker] = rec;
    } else {
        // ---- join the warps through their rings, which are free now
        cp_async_wait_group<0>();
        const int n = cur.n, head0 = first_head(cur);
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
            if (t == 0) s_ml[warp][g + 8 * r] = make_float2(mx[r] - S::LIFT, sum[r]);
        }
        __syncwarp();
        float* const mine = reinterpret_cast<float*>(smem + warp * S::RING);
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int h = 8 * r + 2 * t + (e & 1);
                    const int d = F8 ? 16 * m + 2 * g + (e >> 1) : 16 * m + g + 8 * (e >> 1);
                    mine[h * S::OROW + d] = o[m][r][e];
                }
        __syncthreads();
        const float vs = F8 ? p.v_scale[cur.kvh] : 1.f;
        for (int it = tid; it < heads * (D / 4); it += THREADS) {
            const int h = it / (D / 4), d = (it - h * (D / 4)) * 4;
            const int64_t at = int64_t(n) * p.Hq + head0 + h;
            const float sk = p.sink ? p.sink[at] * kLog2e : -INFINITY;
            float2 ml[WARPS];
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                ml[w] = s_ml[w][h];
                m = fmaxf(m, ml[w].x);
            }
            const float top = fmaxf(m, sk);
            float l = top == -INFINITY ? 0.f : weight(sk, top);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float f = weight(ml[w].x, top);
                const float4 x = *reinterpret_cast<const float4*>(smem + w * S::RING + (h * S::OROW + d) * 4);
                l = fmaf(ml[w].y, f, l);
                acc.x = fmaf(x.x, f, acc.x);
                acc.y = fmaf(x.y, f, acc.y);
                acc.z = fmaf(x.z, f, acc.z);
                acc.w = fmaf(x.w, f, acc.w);
            }
            const float mul = l == 0.f ? 0.f : vs / l;
            *reinterpret_cast<float4*>(p.out + at * D + d) =
                make_float4(acc.x * mul, acc.y * mul, acc.z * mul, acc.w * mul);
            if (d == 0) p.lse[at] = lse_of(m, top, l, p.sink, at);
        }
    }
}

// Joins the parts of each unit that the even split of the tiles cut. Its parts are the
// second slot of the worker that began it and the first slots of the next `more` workers,
// in the order of the keys. Four blocks (blockIdx.z) read the records of 32 workers and take
// query head blockIdx.y of the units that those began and did not finish. Where these are
// one or two, so that their chains of parts may be long, each block takes a quarter of the
// columns and shares the parts out among all its warps and groups of lanes; where they are
// more, each warp takes a unit. All latency, of loads and of the code itself, which is never
// in the caches: so one short kernel.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeParams p,
                                                                   int workers) {
    constexpr int WARPS = kJoinThreads / 32;
    static_assert(WARPS * 4 == 32, "four blocks have a warp for each of 32 workers");
    __shared__ float4 s_acc[WARPS][D / 16];
    __shared__ float2 s_ml[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
    const int w0 = blockIdx.x * 32;
    release_successor();
    wait_for_predecessor();

    int4 rec = make_int4(0, 0, 0, 0);
    if (w0 + lane < workers) rec = *reinterpret_cast<const int4*>(p.rec + w0 + lane);
    uint32_t owners = __ballot_sync(0xffffffffu, rec.w > 0 && h < rec.z);
    const bool together = __popc(owners) <= 2;
    if (!together)
        for (int x = blockIdx.z * WARPS + warp; x > 0; --x) owners &= owners - 1;
    const int lanes = together ? D / 16 : D / 4;  // that hold a part's columns
    const int groups = 32 / lanes * (together ? WARPS : 1), group = lane / lanes + (together ? warp * (32 / lanes) : 0);
    const int column = lane & (lanes - 1), d = (together ? blockIdx.z * (D / 4) : 0) + column * 4;
    for (; owners != 0; owners = together ? owners & (owners - 1) : 0u) {
        const int src = __ffs(owners) - 1;
        const int64_t row = (int64_t(__shfl_sync(0xffffffffu, rec.y, src)) << 32) +
                            uint32_t(__shfl_sync(0xffffffffu, rec.x, src)) + h;
        const int parts = __shfl_sync(0xffffffffu, rec.w, src) + 1;
        const float sk = p.sink ? p.sink[row] * kLog2e : -INFINITY;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float m = -INFINITY, l = 0.f;
        for (int x0 = group; x0 < parts; x0 += kJoinBatch * groups) {
            float2 ml[kJoinBatch];
            float4 y[kJoinBatch];
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                const int x = x0 + k * groups;
                ml[k] = make_float2(-INFINITY, 0.f);
                y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x < parts) {
                    const int64_t at = int64_t(2 * (w0 + src + x) + (x == 0 ? 1 : 0)) * p.unit_heads + h;
                    ml[k] = p.part_ml[at];
                    y[k] = *reinterpret_cast<const float4*>(p.part_o + at * D + d);
                }
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) top = fmaxf(top, ml[k].x);
            const float f = weight(m, top);
            m = top;
            l *= f;
            acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                const float w = weight(ml[k].x, top);
                l = fmaf(ml[k].y, w, l);
                acc = make_float4(fmaf(y[k].x, w, acc.x), fmaf(y[k].y, w, acc.y), fmaf(y[k].z, w, acc.z),
                                  fmaf(y[k].w, w, acc.w));
            }
        }
        auto take = [&](const float2& ml, const float4& y) {  // another group's result
            const float top = fmaxf(m, ml.x), f = weight(m, top), w = weight(ml.x, top);
            m = top;
            l = l * f + ml.y * w;
            acc = make_float4(acc.x * f + y.x * w, acc.y * f + y.y * w, acc.z * f + y.z * w, acc.w * f + y.w * w);
        };
        for (int o = lanes; o < 32; o <<= 1)
            take(make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o)),
                 make_float4(__shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o),
                             __shfl_xor_sync(0xffffffffu, acc.z, o), __shfl_xor_sync(0xffffffffu, acc.w, o)));
        if (together) {
            __syncthreads();
            if (lane < lanes) s_acc[warp][lane] = acc;
            if (lane == 0) s_ml[warp] = make_float2(m, l);
            __syncthreads();
            if (warp != 0) continue;
#pragma unroll 1
            for (int x = 1; x < WARPS; ++x) take(s_ml[x], s_acc[x][column]);
        }
        if (lane >= lanes) continue;
        const float top = fmaxf(m, sk);
        const float f = weight(m, top);
        const float tot = top == -INFINITY ? 0.f : l * f + weight(sk, top);
        const float mul = tot == 0.f ? 0.f : f / tot;
        *reinterpret_cast<float4*>(p.out + row * D + d) =
            make_float4(acc.x * mul, acc.y * mul, acc.z * mul, acc.w * mul);
        if (d == 0) p.lse[row] = lse_of(m, top, tot, p.sink, row);
    }
}

// --------------------------------------------------------------------------
// host
// --------------------------------------------------------------------------
struct Layout {
    size_t rec, ml, o, total;
};
Layout layout_of(int64_t D, int64_t group) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = size_t(2) * kMaxWorkers * (group < 16 ? group : 16);
    Layout l{};
    l.rec = 0;
    l.ml = up(kMaxWorkers * sizeof(Rec));
    l.o = up(l.ml + rows * sizeof(float2));
    l.total = up(l.o + rows * D * 4);
    return l;
}

// Query heads of a unit are 8 or 16, a tile's keys 16 or 32 (Shape).
int64_t units_of(int64_t requests, int64_t heads_kv, int64_t group) {
    return requests * heads_kv * (group <= 8 ? 1 : (group + 15) / 16);
}
int64_t tiles_of(int64_t span, int64_t head_dim, bool e4m3) {
    const int64_t kt = head_dim == 128 && !e4m3 ? 16 : 32;
    return (span + kt - 1) / kt;
}

// Sizes that take the whole form on any device: no workspace is used.
bool never_split(const inkling_kv_cache_desc* c, const inkling_rel_attn_decode_dims* d) {
    int64_t span = d->max_pages * c->page_size;
    if (d->window > 0 && d->window < span) span = d->window;
    return tiles_of(span, c->head_dim, c->dtype == INKLING_KV_E4M3) <= 4 * kWholeTiles &&
           units_of(d->requests, c->heads_kv, d->heads_q / c->heads_kv) <= kWholeUnits;
}

inkling_status check_decode(const inkling_kv_cache_desc* c, const inkling_rel_attn_decode_dims* d, CacheLayout* lay) {
    const inkling_status s = check_cache(c, lay);
    if (s != INKLING_OK) return s;
    if (!d || d->requests < 0 || d->heads_q <= 0 || d->rel_extent < 0 || d->window < 0 || d->max_pages <= 0)
        return INKLING_ERR_INVALID_ARG;
    if (d->heads_q % c->heads_kv != 0 || std::isnan(d->scale) || std::isinf(d->scale)) return INKLING_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 30;
    if (d->requests >= (int64_t(1) << 24) || d->heads_q >= 65536 || d->rel_extent >= lim || d->window >= lim ||
        d->max_pages >= lim || d->max_pages * c->page_size >= lim)
        return INKLING_ERR_UNSUPPORTED;
    if (d->rel_extent % 8 != 0) return INKLING_ERR_UNSUPPORTED;  // profile rows are copied 16 bytes at a time
    // a worker counts its tiles in 32 bits
    if (d->requests * d->heads_q >= (int64_t(1) << 40) / (d->max_pages * c->page_size + 1))
        return INKLING_ERR_UNSUPPORTED;
    return INKLING_OK;
}

inkling_status status_of(cudaError_t e) { return note_cuda_error(e) == cudaSuccess ? INKLING_OK : INKLING_ERR_CUDA; }

// Streaming multiprocessors of a device, looked up once.
cudaError_t sm_count(int dev, int* sms) {
    static std::atomic<int> known[64];
    *sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (*sms != 0) return cudaSuccess;
    const cudaError_t e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
    return e;
}

// The kernel's limit of dynamic shared memory is raised on a device's first launch, and again
// where a launch finds it too low (the device was reset since).
template <class S, int WHOLE>
cudaError_t launch_form(const DecodeParams& p, int64_t grid, int dev, cudaStream_t st) {
    constexpr int warps = WHOLE ? WHOLE : kWarps;
    static std::atomic<uint64_t> raised{0};
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    for (bool again = false;; again = true) {
        if (again || !(raised.load(std::memory_order_relaxed) & bit)) {
            const cudaError_t e = cudaFuncSetAttribute(decode_kernel<S, WHOLE>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, warps * S::RING);
            if (e != cudaSuccess) return e;
            raised.fetch_or(bit, std::memory_order_relaxed);
        }
        const cudaError_t e =
            launch_early(decode_kernel<S, WHOLE>, dim3(unsigned(grid)), 32 * warps, warps * S::RING, st, p);
        if (e != cudaErrorInvalidValue || again) return e;
    }
}

template <class S>
cudaError_t launch_decode(DecodeParams& p, cudaStream_t st) {
    p.hblocks = (p.group + 8 * S::NT - 1) / (8 * S::NT);
    p.unit_heads = p.group < 8 * S::NT ? p.group : 8 * S::NT;
    static_assert(S::KT == (S::D == 128 && !S::F8 ? 16 : 32), "tiles_of");
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = sm_count(dev, &sms);
    if (e != cudaSuccess) return e;
    // at most the tiles of a full table
    const int span = p.W > 0 && p.W < p.cap ? p.W : p.cap;
    const int64_t unit_tiles = tiles_of(span, S::D, S::F8);
    const int64_t units = units_of(p.N, p.Hkv, p.group);
    // eight warps where every unit has an SM to itself and more tiles than four warps
    if (unit_tiles <= 8 * kWholeTiles && unit_tiles > 4 && units <= sms) return launch_form<S, 8>(p, units, dev, st);
    if (unit_tiles <= 4 * kWholeTiles && units <= kWholeUnits) return launch_form<S, 4>(p, units, dev, st);
    const int64_t workers = std::max<int64_t>(units * (unit_tiles + 1) / S::MIN_TILES, 1);
    int64_t grid = int64_t(sms) * kCtasPerSm;
    if (grid > kMaxCtas) grid = kMaxCtas;
    if (grid > (workers + kWarps - 1) / kWarps) grid = (workers + kWarps - 1) / kWarps;
    e = launch_form<S, 0>(p, grid, dev, st);
    if (e != cudaSuccess) return e;
    return launch_early(decode_join_kernel<S::D>,
                        dim3(unsigned((grid * kWarps + 31) / 32), unsigned(p.unit_heads), 4), kJoinThreads, 0, st, p,
                        int(grid) * kWarps);
}

template <int D, bool F8>
cudaError_t launch_group(DecodeParams& p, cudaStream_t st) {
    // one group of 8 query heads per unit where that holds them all, else two: K and V are
    // then read once for up to 16 heads of a group
    return p.group <= 8 ? launch_decode<Shape<D, 1, F8>>(p, st) : launch_decode<Shape<D, 2, F8>>(p, st);
}

}  // namespace

extern "C" {

size_t inkling_rel_attn_decode_workspace_size(const inkling_kv_cache_desc* cache,
                                              const inkling_rel_attn_decode_dims* dims) {
    CacheLayout lay;
    if (check_decode(cache, dims, &lay) != INKLING_OK) return 0;
    if (never_split(cache, dims)) return 256;
    return layout_of(cache->head_dim, dims->heads_q / cache->heads_kv).total;
}

inkling_status inkling_rel_attn_decode(const inkling_kv_cache_desc* cache, const inkling_rel_attn_decode_dims* dims,
                                       const uint16_t* q, const void* k_cache, const void* v_cache,
                                       const float* k_scale, const float* v_scale, const uint16_t* profiles,
                                       const float* sink, const int32_t* block_table, const int32_t* lens, float* out,
                                       float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    NvtxRange nvtx_range("inkling_rel_attn_decode");
    CacheLayout lay;
    const inkling_status s = check_decode(cache, dims, &lay);
    if (s != INKLING_OK) return s;
    if (lay.e4m3 != (k_scale != nullptr) || lay.e4m3 != (v_scale != nullptr)) return INKLING_ERR_INVALID_ARG;
    if ((dims->rel_extent > 0) != (profiles != nullptr)) return INKLING_ERR_INVALID_ARG;
    if (dims->requests == 0) return INKLING_OK;
    if (!q || !k_cache || !v_cache || !block_table || !lens || !out || !lse || !workspace)
        return INKLING_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(profiles, 16) ||
        !aligned(out, 16) || !aligned(workspace, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
        !aligned(sink, 4) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
        return INKLING_ERR_INVALID_ARG;
    const int64_t D = cache->head_dim;
    const Layout l = layout_of(D, dims->heads_q / cache->heads_kv);
    if (workspace_bytes < (never_split(cache, dims) ? 256 : l.total)) return INKLING_ERR_INVALID_ARG;

    DecodeParams p{};
    p.N = int(dims->requests);
    p.Hq = int(dims->heads_q);
    p.Hkv = int(cache->heads_kv);
    p.group = p.Hq / p.Hkv;
    p.R = int(dims->rel_extent);
    p.W = int(dims->window);
    p.M = int(dims->max_pages);
    p.page = PageDivisor(cache->page_size);
    p.num_pages = int(cache->num_pages);
    p.cap = int(dims->max_pages * cache->page_size);
    const int64_t es = lay.e4m3 ? 1 : 2;
    p.page_stride = lay.page_stride * es;
    p.token_stride = lay.token_stride * es;
    p.head_stride = lay.head_stride * es;
    const double scale = dims->scale > 0 ? dims->scale : 1.0 / std::sqrt(double(D));
    p.scale_log2 = std::max(float(scale * 1.4426950408889634), 0x1p-126f);
    p.q = q;
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.profiles = profiles;
    p.sink = sink;
    p.table = block_table;
    p.lens = lens;
    p.out = out;
    p.lse = lse;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.rec = reinterpret_cast<Rec*>(ws + l.rec);
    p.part_ml = reinterpret_cast<float2*>(ws + l.ml);
    p.part_o = reinterpret_cast<float*>(ws + l.o);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (D == 128) return status_of(lay.e4m3 ? launch_group<128, true>(p, st) : launch_group<128, false>(p, st));
    return status_of(lay.e4m3 ? launch_group<64, true>(p, st) : launch_group<64, false>(p, st));
}

}  // extern "C"
