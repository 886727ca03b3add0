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
//   * the grid is two CTAs of four warps per SM, whatever the batch; all CTA tiles (4 warps
//     x KT keys) of all (request, KV head) units are numbered through and each CTA takes an
//     equal run of them, so ragged batches and single long requests load every SM the same.
//     The run is found on the device from the lengths: nothing about them is needed on the
//     host. A unit that is cut leaves its parts in the workspace and a second kernel,
//     launched while the first one runs, joins them in the order of the keys.
//   * each warp streams tiles of its own through a private cp.async ring in shared memory
//     (no block barrier inside a unit) and keeps its own m, l and O; the four are joined
//     once per unit. cp.async with one row address per key takes any page size and any
//     strides, and fills the rows of keys that are not allowed with zeros, so nothing that
//     stands in such a place (NaN, infinities) reaches a product.
//   * products are mma.sync m16n8k16: with a group of 8 heads or fewer a tile is far too
//     narrow for tcgen05 (64 or 128 rows of M), and the tensor pipe is idle most of the
//     time anyway. S[heads, keys] = Q K^T puts the heads in M, so its accumulators are
//     already the B operand of O^T[d, heads] = V^T P^T: no shuffle between the products.
//     K fragments come by ldmatrix, V fragments by its transposing form.
//   * probabilities enter the second product as the sum of two 16-bit numbers (p and what
//     its rounding left), which costs one more mma on an idle pipe and keeps the FP32
//     result to about 2^-18 of a probability instead of 2^-9.
// e4m3 caches: a code is exact in FP16, so both products run in FP16 with FP32 sums; the
// scales stay outside the products. q (BF16) is first multiplied by a power of two per
// head that brings its largest value into [1, 2): exact but for values below 2^-14 of
// the largest, whose error (2^-25 of it) is under the FP32 sum's own.
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
constexpr int kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 320;  // workspace slots: two per CTA
constexpr int kMaxHeads = 16;  // query heads of a unit at most

struct Rec {  // what a CTA's last unit left unfinished: parts 1 .. more are in the next CTAs
    int n, u, more, pad;
};

struct DecodeParams {
    int N, Hq, Hkv, group, hblocks, R, W, M, P, num_pages, cap;
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
    Rec* rec;          // [grid]
    float2* part_ml;   // [2 * grid][kMaxHeads]
    float* part_o;     // [2 * grid][kMaxHeads][D]
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

// two e4m3 codes (low and high byte) as an FP16 pair, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(codes)));
    return r;
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
// cache. A tile is 8 KB of K and V in every form but the smallest, so that three of them
// per warp are 64 KB or more in flight on an SM.
template <int D_, int NT_, bool F8_>
struct Shape {
    static constexpr int D = D_, NT = NT_;
    static constexpr bool F8 = F8_;
    static constexpr int ES = F8 ? 1 : 2;
    static constexpr int RB = D * ES;                    // bytes of a row
    static constexpr int CPR = RB / 16;                  // 16-byte chunks of a row
    static constexpr int KT = (D == 128 && !F8) ? 16 : 32;  // keys of a warp's tile
    static constexpr int CT = kWarps * KT;               // keys of a CTA tile
    static constexpr int STAGES = 3;
    static constexpr int SIDE = KT * RB;                 // bytes of K (or V) in a stage
    static constexpr int RING = STAGES * 2 * SIDE;       // bytes of a warp's ring
    static constexpr int OROW = D + 4;                   // floats of a head's row in the join (no bank conflicts)
    static constexpr int REGION = RING > 8 * NT * OROW * 4 ? RING : 8 * NT * OROW * 4;  // the join reuses the ring
    static constexpr int SMEM = kWarps * REGION;
    __device__ static __forceinline__ int swz(int row) { return RB >= 128 ? (row & 7) : ((row >> 1) & 3); }
};

struct Span {  // allowed keys [lo, len) of a request and its CTA tiles (at least one)
    int lo, len, tiles;
};
template <int CT>
__device__ __forceinline__ Span span_of(const DecodeParams& p, int n) {
    Span s;
    s.len = min(max(p.lens[n], 0), p.cap);
    s.lo = p.W > 0 ? max(s.len - p.W, 0) : 0;
    s.tiles = max((s.len - s.lo + CT - 1) / CT, 1);
    return s;
}

// lse of a row from the maximum of its keys' logits, that of those and the sink (log2 units),
// and the sum over both relative to it; the sink itself where no key is left.
__device__ __forceinline__ float lse_of(float keys, float top, float total, const float* sink, int64_t at) {
    if (keys == -INFINITY && total <= 1.f) return sink ? sink[at] : -INFINITY;
    return (top + log2f(total)) * kLn2;
}

template <class S>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_kernel(const DecodeParams p) {
    constexpr int D = S::D, NT = S::NT, KT = S::KT, ST = S::STAGES;
    constexpr bool F8 = S::F8;
    constexpr int NS = KT / 8;  // S accumulator tiles of 8 keys
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t s_mask[kWarps][ST];
    __shared__ float2 s_ml[kWarps][8 * NT];
    __shared__ long long s_sum[kWarps];
    __shared__ long long s_base;
    __shared__ int s_n;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    // the joining kernel may be set up now; it waits for this one's results itself
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- this CTA's run of tiles
    const int64_t units = int64_t(p.Hkv) * p.hblocks;  // per request
    const int chunk = (p.N + kThreads - 1) / kThreads;
    const int n0 = min(tid * chunk, p.N), n1 = min(n0 + chunk, p.N);
    long long own = 0;
    for (int n = n0; n < n1; ++n) own += span_of<S::CT>(p, n).tiles;
    long long inc = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += x;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    long long before = inc - own, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        all += s_sum[w];
    }
    all *= units;
    const int ctas = int(all < gridDim.x ? all : (long long)gridDim.x);
    const int cta = blockIdx.x;
    if (cta >= ctas) {
        if (tid == 0) p.rec[cta] = Rec{0, 0, 0, 0};
        return;
    }
    const long long first = cta * all / ctas, last = (cta + 1) * all / ctas;
    if (before * units <= first && first < (before + own) * units) {
        long long at = before * units;
        int n = n0;
        for (;; ++n) {
            const long long size = span_of<S::CT>(p, n).tiles * units;
            if (first < at + size) break;
            at += size;
        }
        s_n = n;
        s_base = at;
    }
    __syncthreads();
    int n = s_n;
    long long base = s_base;

    const uint32_t ring = smem_u32(smem) + warp * S::REGION;
    const float* const ofloat = reinterpret_cast<const float*>(smem);
    Rec rec{0, 0, 0, 0};

    for (long long pos = first; pos < last;) {
        const Span sp = span_of<S::CT>(p, n);
        const long long local = pos - base;
        const int u = int(local / sp.tiles), tile0 = int(local - (long long)u * sp.tiles);
        const long long room = last - pos;
        const int tile1 = int(sp.tiles - tile0 < room ? sp.tiles : tile0 + room);
        const int kvh = u / p.hblocks, hb = u - kvh * p.hblocks;
        const int head0 = kvh * p.group + hb * 8 * NT;
        const int heads = min(8 * NT, p.group - hb * 8 * NT);
        const int nt = tile1 - tile0;  // tiles of each warp
        const int key_end = min((long long)sp.len, sp.lo + (long long)tile1 * S::CT);
        const int key0 = sp.lo + tile0 * S::CT + warp * KT;  // first key of this warp's tile 0; step CT
        const int32_t* const row = p.table + int64_t(n) * p.M;

        // ---- q fragments
        uint32_t qa[D / 16][2 * NT];
        float zscale[NT];
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            const int h = g + 8 * r;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + (int64_t(n) * p.Hq + head0 + h) * D);
            zscale[r] = p.scale_log2;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                // BF16: columns 16 ks + {2t, 2t+1} and + 8; e4m3: 16 ks + {4t .. 4t+3}, the
                // order in which a code word holds them (K uses the same one)
                const int w0 = F8 ? 8 * ks + 2 * t : 8 * ks + t, w1 = F8 ? w0 + 1 : w0 + 4;
                qa[ks][2 * r] = h < heads ? src[w0] : 0u;
                qa[ks][2 * r + 1] = h < heads ? src[w1] : 0u;
            }
            if constexpr (F8) {
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = unpack2<false>(qa[ks][2 * r + i]);
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
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = unpack2<false>(qa[ks][2 * r + i]);
                        qa[ks][2 * r + i] = pack2<true>(x.x * down, x.y * down);
                    }
                zscale[r] *= __uint_as_float(uint32_t(127 + e) << 23) * p.k_scale[kvh];
            }
        }

        float o[D / 16][NT][4];
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][x][i] = 0.f;
        float mx[NT], sum[NT];
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            mx[r] = -INFINITY;
            sum[r] = 0.f;
        }

        // ---- producer: lane r < KT looks key r of a tile up, all lanes copy
        const int my_key = lane & (KT - 1);
        auto page_of = [&](int i) {  // -1: not allowed
            const int j = key0 + i * S::CT + my_key;
            return i < nt && j < key_end ? row[j / p.P] : -1;
        };
        auto issue = [&](int i, int stage, int page) {
            const int j = key0 + i * S::CT + my_key;
            const bool ok = page >= 0 && page < p.num_pages;
            const uint32_t mask = __ballot_sync(0xffffffffu, ok);
            if (lane == 0) s_mask[warp][stage] = mask;
            const int64_t at =
                ok ? int64_t(page) * p.page_stride + int64_t(j % p.P) * p.token_stride + kvh * p.head_stride : 0;
            const uint32_t dst = ring + stage * 2 * S::SIDE;
#pragma unroll
            for (int c = 0; c < KT * S::CPR / 32; ++c) {
                const int r = c * (32 / S::CPR) + lane / S::CPR, ch = lane % S::CPR;
                const int64_t off = __shfl_sync(0xffffffffu, at, r) + ch * 16;
                const uint32_t bytes = (mask >> r) & 1u ? 16u : 0u;
                const uint32_t to = dst + r * S::RB + ((ch ^ S::swz(r)) << 4);
                cp_async_16(to, p.k_cache + off, bytes);
                cp_async_16(to + S::SIDE, p.v_cache + off, bytes);
            }
        };
        // ---- bias of this thread's S entries of tile i (BF16 bits, 0 beyond the profile)
        const bool biased = p.R > 0;
        uint16_t bias[NT][NS][2];
        auto load_bias = [&](int i) {
            const int j0 = key0 + i * S::CT;
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int s = 0; s < NS; ++s) bias[r][s][0] = bias[r][s][1] = 0;
            if (!biased || i >= nt || sp.len - 1 - (j0 + KT - 1) >= p.R) return;
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                if (g + 8 * r >= heads) continue;
                const uint16_t* prof = p.profiles + (int64_t(n) * p.Hq + head0 + g + 8 * r) * p.R;
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = sp.len - 1 - (j0 + 8 * s + 2 * t + e);
                        if (d >= 0 && d < p.R) bias[r][s][e] = __ldg(prof + d);
                    }
            }
        };

        int page = -1;
        {
            int first_pages[ST - 1];
#pragma unroll
            for (int i = 0; i < ST - 1; ++i) first_pages[i] = page_of(i);
            page = page_of(ST - 1);
#pragma unroll
            for (int i = 0; i < ST - 1; ++i) {
                if (i < nt) issue(i, i, first_pages[i]);
                cp_async_commit();
            }
        }
        load_bias(0);

        int stage = 0;
        for (int i = 0; i < nt; ++i) {
            cp_async_wait_group<ST - 2>();
            __syncwarp();  // the tile is in, and every lane is done with the previous one's stage
            {
                const int next = i + ST - 1;
                const int to = stage == 0 ? ST - 1 : stage - 1;
                if (next < nt) issue(next, to, page);
                cp_async_commit();
                page = page_of(next + 1);
            }
            uint16_t b_now[NT][NS][2];
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    b_now[r][s][0] = bias[r][s][0];
                    b_now[r][s][1] = bias[r][s][1];
                }
            load_bias(i + 1);

            const uint32_t mask = s_mask[warp][stage];
            const uint32_t kbase = ring + stage * 2 * S::SIDE, vbase = kbase + S::SIDE;
            stage = stage == ST - 1 ? 0 : stage + 1;
            if (mask == 0) continue;

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
                        const uint32_t a1 = NT == 2 ? qa[c][2 * (NT - 1)] : 0u, a3 = NT == 2 ? qa[c][2 * NT - 1] : 0u;
                        mma16816<false>(s[2 * kk], qa[c][0], a1, qa[c][1], a3, f[0], f[1]);
                        mma16816<false>(s[2 * kk + 1], qa[c][0], a1, qa[c][1], a3, f[2], f[3]);
                    } else {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {  // the pair's two chunks: 16 columns each
                            const uint32_t* a = qa[2 * c + x];
                            const uint32_t a1 = NT == 2 ? a[2 * (NT - 1)] : 0u, a3 = NT == 2 ? a[2 * NT - 1] : 0u;
                            mma16816<true>(s[2 * kk], a[0], a1, a[1], a3, e4m3x2_to_f16x2(f[x]),
                                           e4m3x2_to_f16x2(f[x] >> 16));
                            mma16816<true>(s[2 * kk + 1], a[0], a1, a[1], a3, e4m3x2_to_f16x2(f[x + 2]),
                                           e4m3x2_to_f16x2(f[x + 2] >> 16));
                        }
                    }
                }
            }

            // ---- logits in log2 units, their maximum, the running state
            float top[NT];
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                top[r] = -INFINITY;
#pragma unroll
                for (int x = 0; x < NS; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float z = s[x][2 * r + e] * zscale[r];
                        z = fmaf(__uint_as_float(uint32_t(b_now[r][x][e]) << 16), kLog2e, z);
                        if (!((mask >> (8 * x + 2 * t + e)) & 1u)) z = -INFINITY;
                        s[x][2 * r + e] = z;
                        top[r] = fmaxf(top[r], z);
                    }
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            }
            bool grows = false;
#pragma unroll
            for (int r = 0; r < NT; ++r) grows |= top[r] > mx[r] + kRescaleThreshold;
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int r = 0; r < NT; ++r) {
                    const float now = fmaxf(mx[r], top[r]);
                    const float f = mx[r] == now ? 1.f : ex2_approx(mx[r] - now);
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
            uint32_t hi[NT][NS], lo[NT][NS];
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                const float ref = mx[r] == -INFINITY ? 0.f : mx[r];
#pragma unroll
                for (int x = 0; x < NS; ++x) {
                    const float p0 = ex2_approx(s[x][2 * r] - ref), p1 = ex2_approx(s[x][2 * r + 1] - ref);
                    sum[r] += p0 + p1;
                    hi[r][x] = pack2<F8>(p0, p1);
                    const float2 b = unpack2<F8>(hi[r][x]);
                    lo[r][x] = pack2<F8>(p0 - b.x, p1 - b.y);
                }
            }

            // ---- O^T += V^T P^T
#pragma unroll
            for (int c = 0; c < S::CPR / 2; ++c) {
#pragma unroll
                for (int kk = 0; kk < KT / 16; ++kk) {
                    uint32_t f[4];
                    ldmatrix_x4_trans(vbase + (kk * 16 + lrow) * S::RB + (((2 * c + lch) ^ lswz) << 4), f);
                    if constexpr (!F8) {
#pragma unroll
                        for (int r = 0; r < NT; ++r) {
                            mma16816<false>(o[c][r], f[0], f[1], f[2], f[3], hi[r][2 * kk], hi[r][2 * kk + 1]);
                            mma16816<false>(o[c][r], f[0], f[1], f[2], f[3], lo[r][2 * kk], lo[r][2 * kk + 1]);
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            // a 16-bit unit holds columns 2g, 2g + 1 of one key: regroup by column
                            const uint32_t w0 = __byte_perm(f[x], 0, 0x3120), w1 = __byte_perm(f[x + 2], 0, 0x3120);
                            const uint32_t a0 = e4m3x2_to_f16x2(w0), a1 = e4m3x2_to_f16x2(w0 >> 16);
                            const uint32_t a2 = e4m3x2_to_f16x2(w1), a3 = e4m3x2_to_f16x2(w1 >> 16);
#pragma unroll
                            for (int r = 0; r < NT; ++r) {
                                mma16816<true>(o[2 * c + x][r], a0, a1, a2, a3, hi[r][2 * kk], hi[r][2 * kk + 1]);
                                mma16816<true>(o[2 * c + x][r], a0, a1, a2, a3, lo[r][2 * kk], lo[r][2 * kk + 1]);
                            }
                        }
                    }
                }
            }
        }
        cp_async_wait_group<0>();

        // ---- join the four warps (their rings are free now)
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
            if (t == 0) s_ml[warp][g + 8 * r] = make_float2(mx[r], sum[r]);
        }
        __syncwarp();
        float* const mine = reinterpret_cast<float*>(smem + warp * S::REGION);
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int h = 8 * r + 2 * t + (i & 1);
                    const int d = F8 ? 16 * m + 2 * g + (i >> 1) : 16 * m + g + 8 * (i >> 1);
                    mine[h * S::OROW + d] = o[m][r][i];
                }
        __syncthreads();
        const bool starts = tile0 == 0, ends = tile1 == sp.tiles;
        const int slot = 2 * cta + (starts ? 1 : 0);
        const float vs = F8 ? p.v_scale[kvh] : 1.f;
        for (int it = tid; it < heads * (D / 4); it += kThreads) {
            const int h = it / (D / 4), d = (it - h * (D / 4)) * 4;
            float2 ml[kWarps];
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = s_ml[w][h];
                m = fmaxf(m, ml[w].x);
            }
            float l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ml[w].x == m ? 1.f : ex2_approx(ml[w].x - m);
                const float4 x =
                    *reinterpret_cast<const float4*>(ofloat + w * (S::REGION / 4) + h * S::OROW + d);
                l = fmaf(ml[w].y, f, l);
                acc.x = fmaf(x.x, f, acc.x);
                acc.y = fmaf(x.y, f, acc.y);
                acc.z = fmaf(x.z, f, acc.z);
                acc.w = fmaf(x.w, f, acc.w);
            }
            float mul = vs;
            float* to;
            const int64_t at = int64_t(n) * p.Hq + head0 + h;
            if (starts && ends) {
                const float sk = p.sink ? p.sink[at] * kLog2e : -INFINITY;
                const float top = fmaxf(m, sk);
                const float f = m == top ? 1.f : ex2_approx(m - top);
                const float tot = l * f + (sk == top ? (top == -INFINITY ? 0.f : 1.f) : ex2_approx(sk - top));
                mul = tot == 0.f ? 0.f : vs * f / tot;
                to = p.out + at * D + d;
                if (d == 0) p.lse[at] = lse_of(m, top, tot, p.sink, at);
            } else {
                to = p.part_o + (int64_t(slot) * kMaxHeads + h) * D + d;
                if (d == 0) p.part_ml[int64_t(slot) * kMaxHeads + h] = make_float2(m, l);
            }
            *reinterpret_cast<float4*>(to) = make_float4(acc.x * mul, acc.y * mul, acc.z * mul, acc.w * mul);
        }
        if (starts && !ends) {
            const long long unit_end = base + (long long)(u + 1) * sp.tiles;  // first tile behind the unit
            rec = Rec{n, u, int((unit_end * ctas - 1) / all) - cta, 0};
        }
        pos += nt;
        if (pos == base + units * sp.tiles) {
            base = pos;
            ++n;
        }
        __syncthreads();  // the rings may be written again
    }
    if (tid == 0) p.rec[cta] = rec;
}

// Joins the parts of each unit that the tiles' even split cut: block (c, h) takes query
// head h of the unit that CTA c began and did not finish; its other parts are the first
// ones of CTAs c + 1 .. c + more. Parts are added in the order of the keys.
template <int D>
__global__ void __launch_bounds__(D) decode_join_kernel(const DecodeParams p, int block_heads) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x, h = blockIdx.y, d = threadIdx.x;
    const Rec rec = p.rec[c];
    if (rec.more == 0) return;
    const int kvh = rec.u / p.hblocks, hb = rec.u - kvh * p.hblocks;
    if (hb * block_heads + h >= p.group) return;
    auto slot = [&](int i) { return int64_t(i == 0 ? 2 * c + 1 : 2 * (c + i)) * kMaxHeads + h; };
    const int64_t at = int64_t(rec.n) * p.Hq + kvh * p.group + hb * block_heads + h;
    const float sk = p.sink ? p.sink[at] * kLog2e : -INFINITY;
    float keys = -INFINITY;
    for (int i = 0; i <= rec.more; ++i) keys = fmaxf(keys, p.part_ml[slot(i)].x);
    const float m = fmaxf(keys, sk);
    float l = sk == m ? (m == -INFINITY ? 0.f : 1.f) : ex2_approx(sk - m);
    float acc = 0.f;
#pragma unroll 4
    for (int i = 0; i <= rec.more; ++i) {
        const float2 ml = p.part_ml[slot(i)];
        const float f = ml.x == m ? 1.f : ex2_approx(ml.x - m);
        l = fmaf(ml.y, f, l);
        acc = fmaf(p.part_o[slot(i) * D + d], f, acc);
    }
    p.out[at * D + d] = l == 0.f ? 0.f : acc / l;
    if (d == 0) p.lse[at] = lse_of(keys, m, l, p.sink, at);
}

// --------------------------------------------------------------------------
// host
// --------------------------------------------------------------------------
struct Layout {
    size_t rec, ml, o, total;
};
Layout layout_of(int64_t D) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Layout l{};
    l.rec = 0;
    l.ml = up(kMaxCtas * sizeof(Rec));
    l.o = up(l.ml + size_t(2) * kMaxCtas * kMaxHeads * sizeof(float2));
    l.total = up(l.o + size_t(2) * kMaxCtas * kMaxHeads * D * 4);
    return l;
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
    // the tiles are numbered through in 64 bits, times the CTAs
    if (d->requests * d->heads_q >= (int64_t(1) << 50) / (d->max_pages * c->page_size + 1))
        return INKLING_ERR_UNSUPPORTED;
    return INKLING_OK;
}

inkling_status status_of(cudaError_t e) { return note_cuda_error(e) == cudaSuccess ? INKLING_OK : INKLING_ERR_CUDA; }

template <class S>
cudaError_t launch_decode(DecodeParams& p, cudaStream_t st) {
    p.hblocks = (p.group + 8 * S::NT - 1) / (8 * S::NT);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decode_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    // at most the tiles of a full table
    const int span = p.W > 0 && p.W < p.cap ? p.W : p.cap;
    const int64_t unit_tiles = (span + S::CT - 1) / S::CT;
    const int64_t tiles = int64_t(p.N) * p.Hkv * p.hblocks * unit_tiles;
    int64_t grid = int64_t(sms) * kCtasPerSm;
    if (grid > kMaxCtas) grid = kMaxCtas;
    if (grid > tiles) grid = tiles;
    decode_kernel<S><<<unsigned(grid), kThreads, S::SMEM, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || unit_tiles == 1) return e;  // units of one tile are never cut
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(grid), 8 * S::NT < p.group ? 8 * S::NT : p.group);
    cfg.blockDim = dim3(S::D);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_join_kernel<S::D>, DecodeParams(p), 8 * S::NT);
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
    return layout_of(cache->head_dim).total;
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
    const Layout l = layout_of(D);
    if (workspace_bytes < l.total) return INKLING_ERR_INVALID_ARG;

    DecodeParams p{};
    p.N = int(dims->requests);
    p.Hq = int(dims->heads_q);
    p.Hkv = int(cache->heads_kv);
    p.group = p.Hq / p.Hkv;
    p.R = int(dims->rel_extent);
    p.W = int(dims->window);
    p.M = int(dims->max_pages);
    p.P = int(cache->page_size);
    p.num_pages = int(cache->num_pages);
    p.cap = int(dims->max_pages * cache->page_size);
    const int64_t es = lay.e4m3 ? 1 : 2;
    p.page_stride = lay.page_stride * es;
    p.token_stride = lay.token_stride * es;
    p.head_stride = lay.head_stride * es;
    const double scale = dims->scale > 0 ? dims->scale : 1.0 / std::sqrt(double(D));
    p.scale_log2 = float(scale * 1.4426950408889634);
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
