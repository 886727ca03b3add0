// paged_cache.cu -- the paged key-value cache of the serving path
// (include/inkling_paged_attn.h): the page plan of a step and the append of new rows,
// with their C entry points.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "inkling_paged_attn.h"
#include "paged.h"

namespace {

using namespace ira;

// --------------------------------------------------------------------------
// inkling_kv_plan
// --------------------------------------------------------------------------
struct PlanParams {
    int N, M, num_pages, T;
    PageDivisor page;
    const int32_t* old_lens;
    const int32_t* new_lens;
    int32_t* table;
    int32_t* free_pages;
    const int32_t* free_count;
    int32_t* lens;
    int32_t* query_start;
    int64_t* slots;
    int32_t* positions;
    int32_t* info;
};

constexpr int kPlanThreads = 1024;
constexpr int64_t kPlanMaxRequests = 16384;
constexpr size_t kPlanStatic = 32 * sizeof(int3);  // shared memory of plan_kernel beside the prefix sums

__device__ __forceinline__ int pages_of(int len, const PageDivisor& page) {
    return len > 0 ? page.index(len - 1) + 1 : 0;
}

// Largest r in [0, n) with at[r] <= x, for a non-decreasing at with at[0] = 0 <= x.
__device__ __forceinline__ int last_at_or_below(const int* at, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The plan is three prefix sums over the requests (new tokens, pages to take, pages to
// give back) and then independent writes: each new token, taken page, returned page and
// request is an item of its own, and finds its request by bisection. Bound by launch and
// load latency (a few microseconds of work), so it is one kernel with no exchange between
// blocks, all items side by side: every block computes the three sums itself (N <= 16384
// lengths, from L2 after the first block) into shared memory and takes its share of the
// items. The stack needs no order between blocks either: a page popped in the same call that
// returned it is read from the block table, so no block reads an entry of free_pages or of
// the table that another one writes. The code is kept short: it is as cold as the data.
// GPU time: 64 requests of one token each 3.1 us, 256 prompts (239,480 tokens) 5.3 us, 4096
// requests (117,153 tokens) 8.5 us, 8192 (233,359) 19.8 us, 16384 (464,073) 59.6 us: from 4096
// requests on the sums' shared-memory bank conflicts count (a thread's requests stand next to
// each other, so its neighbours are 4, 8 or 16 words away: 429,352 conflicts at 4096, 3,460
// cycles of each block).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams p) {
    extern __shared__ int s_at[];
    int* s_tok = s_at;               // [N + 1] exclusive prefix sums, totals at [N]
    int* s_need = s_tok + p.N + 1;
    int* s_back = s_need + p.N + 1;
    __shared__ int3 s_warp[kPlanStatic / sizeof(int3)];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // no early release: blocks of a successor that come in beside these share their SMs unevenly
    // (two plans of 4096 requests in a row 13.5 us each instead of 9.0)
    wait_for_predecessor();
    const int free_count = *p.free_count;  // plain loads: see wait_for_predecessor
    const int cap = p.M * p.page.size;
    auto old_len = [&](int r) { return min(max(p.old_lens[r], 0), cap); };
    auto new_len = [&](int r) { return min(max(p.new_lens[r], 0), cap); };

    const int chunk = (p.N + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(tid * chunk, p.N), r1 = min(r0 + chunk, p.N);
    int3 sum = make_int3(0, 0, 0);
    for (int first = r0; first < r1; first += 4) {  // four requests' loads ahead of the stores
        int o[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] = first + i < r1 ? old_len(first + i) : 0;
            w[i] = first + i < r1 ? new_len(first + i) : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (first + i >= r1) break;
            const int held = pages_of(o[i], p.page), want = pages_of(w[i], p.page);
            s_tok[first + i] = sum.x;
            s_need[first + i] = sum.y;
            s_back[first + i] = sum.z;
            sum.x += max(w[i] - o[i], 0);
            sum.y += max(want - held, 0);
            sum.z += max(held - want, 0);
        }
    }
    auto scan = [&](int3 v) {  // inclusive, over the warp
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, v.x, d), y = __shfl_up_sync(0xffffffffu, v.y, d),
                      z = __shfl_up_sync(0xffffffffu, v.z, d);
            if (lane >= d) v = make_int3(v.x + x, v.y + y, v.z + z);
        }
        return v;
    };
    const int3 inc = scan(sum);
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    const int3 warps = scan(lane < kPlanThreads / 32 ? s_warp[lane] : make_int3(0, 0, 0));
    const int3 all = make_int3(__shfl_sync(0xffffffffu, warps.x, 31), __shfl_sync(0xffffffffu, warps.y, 31),
                               __shfl_sync(0xffffffffu, warps.z, 31));
    const int prev = max(warp - 1, 0);
    int3 ex = make_int3(__shfl_sync(0xffffffffu, warps.x, prev), __shfl_sync(0xffffffffu, warps.y, prev),
                        __shfl_sync(0xffffffffu, warps.z, prev));
    if (warp == 0) ex = make_int3(0, 0, 0);
    ex = make_int3(ex.x + inc.x - sum.x, ex.y + inc.y - sum.y, ex.z + inc.z - sum.z);
    for (int r = r0; r < r1; ++r) {
        s_tok[r] += ex.x;
        s_need[r] += ex.y;
        s_back[r] += ex.z;
    }
    if (tid == 0) {
        s_tok[p.N] = all.x;
        s_need[p.N] = all.y;
        s_back[p.N] = all.z;
    }
    __syncthreads();

    const int count = min(max(free_count, 0), p.num_pages);
    // returned pages beyond the stack's room (malformed tables only) are dropped
    const int back = min(all.z, p.num_pages - count);
    const int avail = count + back;
    const int taken = min(all.y, avail);
    const int left = avail - taken;
    const int kept = min(back, max(left - count, 0));  // returned pages that this call does not pop again

    auto returned = [&](int i) {
        const int r = last_at_or_below(s_back, p.N, i);
        return p.table[int64_t(r) * p.M + pages_of(new_len(r), p.page) + (i - s_back[r])];
    };
    auto popped = [&](int k) {
        const int at = avail - 1 - k;
        return at < count ? p.free_pages[at] : returned(at - count);
    };

    const int64_t items = int64_t(p.T) + taken + kept + p.N + 1;
    for (int64_t item = int64_t(blockIdx.x) * kPlanThreads + tid; item < items; item += gridDim.x * kPlanThreads) {
        if (item < int64_t(p.T) + taken) {  // a token, or a page taken
            const bool token = item < p.T;
            const int i = int(token ? item : item - p.T);
            int64_t slot = -1;
            int pos = 0;
            if (!token || i < all.x) {
                const int* at = token ? s_tok : s_need;
                const int r = last_at_or_below(at, p.N, i);
                const int o = old_len(r), held = pages_of(o, p.page);
                pos = o + (i - at[r]);
                const int idx = token ? p.page.index(pos) : held + (i - at[r]);
                const int k = s_need[r] + (idx - held);
                int page = -1;
                if (idx < held) page = p.table[int64_t(r) * p.M + idx];
                else if (k < taken) page = popped(k);
                if (!token) p.table[int64_t(r) * p.M + idx] = page;
                if (page >= 0 && page < p.num_pages) slot = int64_t(page) * p.page.size + (pos - idx * p.page.size);
            }
            if (token) {
                p.slots[i] = slot;
                p.positions[i] = pos;
            }
        } else if (item < int64_t(p.T) + taken + kept) {
            const int i = int(item - p.T - taken);
            p.free_pages[count + i] = returned(i);
        } else {
            const int r = int(item - p.T - taken - kept);
            p.query_start[r] = s_tok[r];
            if (r == p.N) {
                p.info[0] = left;
                p.info[1] = all.x;
                p.info[2] = all.y - taken;
                p.info[3] = taken;
            } else {
                const int o = old_len(r), w = new_len(r);
                const int64_t given = min(max(taken - s_need[r], 0), s_need[r + 1] - s_need[r]);
                const int64_t room = (pages_of(o, p.page) + given) * p.page.size;
                p.lens[r] = w <= o ? w : int(room < w ? room : w);
            }
        }
    }
}

inkling_status check_plan(const inkling_kv_plan_dims* d) {
    if (!d) return INKLING_ERR_INVALID_ARG;
    if (d->requests < 0 || d->page_size <= 0 || d->max_pages <= 0 || d->num_pages <= 0 || d->max_tokens < 0)
        return INKLING_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 30;
    if (d->requests > kPlanMaxRequests || d->page_size >= lim || d->max_pages >= lim || d->num_pages > 0x7fffffff ||
        d->max_tokens > lim)
        return INKLING_ERR_UNSUPPORTED;
    const int64_t cap = d->max_pages * d->page_size;
    if (cap >= (int64_t(1) << 31) || cap * (d->requests ? d->requests : 1) >= (int64_t(1) << 31))
        return INKLING_ERR_UNSUPPORTED;
    return INKLING_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

// --------------------------------------------------------------------------
// inkling_kv_append
// --------------------------------------------------------------------------
struct AppendParams {
    unsigned rows;  // T * Hkv
    PageDivisor heads, page;
    int64_t num_slots, page_stride, token_stride, head_stride, k_row, v_row;
    float thr;
    const uint16_t* k;
    const uint16_t* v;
    const int64_t* slots;
    const float* k_scale;
    const float* v_scale;
    const float* clip_scale;
    const float* tau;
    void* k_cache;
    void* v_cache;
};

constexpr int kAppendThreads = 128;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// x / scale, saturated and rounded to nearest even. The quotient is the correctly rounded
// one, so that the codes are those of the formula at every tie: with y the reciprocal of the
// scale rounded to nearest, q = x y is corrected once by its remainder (Markstein's division:
// both steps are fused multiply-adds; this order of the signs keeps that of a zero).
// Infinities have no remainder, and with a scale below 2^-60 or above 2^60 it could leave the
// normal numbers: those eight values divide.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
    const float y = __frcp_rn(scale);
    float q[8], top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = x[i] * y;
        top = fmaxf(top, fabsf(q[i]));
    }
    if (top < INFINITY && scale > 0x1p-60f && scale < 0x1p60f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = fmaf(-fmaf(q[i], scale, -x[i]), y, q[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], scale);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Values of a row that a lane takes: 16 bytes of the cache's type.
template <bool E4M3>
constexpr int kPerLane = E4M3 ? 16 : 8;

// One (token, head) row of k and of v per group of lanes, 16-byte loads and one 16-byte store
// of each to a lane, all rows of a token next to each other. A stream of 4 (BF16) or 3
// (e4m3) bytes per value, bound by HBM; the clipped e4m3 form by how many threads an SM holds
// and by its arithmetic between loads and stores (61 % of the issue slots busy; 77 % with 8
// values to a lane, which is why a lane has 16). No loop, so that a full SM keeps the loads of
// all its threads in flight: 2048 in BF16 (18 and 32 registers), 1536 and, clipped, 1280 in
// e4m3 (40 and 48). The clip's sum of squares is FP32 over the group by shuffles.
// 32768 clipped rows of 8 x 128: 42.1 us, 6.39 TB/s; 16381 clipped rows of 4 x 128 to e4m3
// 11.4 us, 4.4 TB/s, unclipped 8.4 us, 6.0 TB/s; one step of 64 rows: 1.3 us. (128 threads to a
// block: with 256, 11.6 and 1.5 us; held to fewer registers, the clipped e4m3 form spills and
// takes 12.9 us and more.)
template <int D, bool E4M3, bool CLIP>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int PER = kPerLane<E4M3>, LPR = D / PER;
    release_successor();
    wait_for_predecessor();
    const unsigned row = blockIdx.x * (kAppendThreads / LPR) + threadIdx.x / LPR;
    const int at_d = threadIdx.x % LPR * PER;
    const unsigned t = p.heads.index(row), g = row - t * p.heads.size;
    const uint32_t peers = __ballot_sync(0xffffffffu, row < p.rows);
    if (row >= p.rows) return;  // whole groups leave together
    // every load at once: a row that is skipped in the end is read too
    const int64_t slot = p.slots[t];
    const uint4* const kp = reinterpret_cast<const uint4*>(p.k + t * p.k_row + g * D + at_d);
    const uint4* const vp = reinterpret_cast<const uint4*>(p.v + t * p.v_row + g * D + at_d);
    uint4 ku[PER / 8], vu[PER / 8];
#pragma unroll
    for (int i = 0; i < PER / 8; ++i) {
        ku[i] = __ldcs(kp + i);
        vu[i] = __ldcs(vp + i);
    }
    float ks = 1.f, vs = 1.f;
    if constexpr (E4M3) {
        ks = p.k_scale[g];
        vs = p.v_scale[g];
    }
    if constexpr (CLIP) {
        const float tau = p.tau ? p.tau[t] : 1.f;
        float kx[PER / 8][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < PER / 8; ++i) {
            unpack8(ku[i], kx[i]);
            if (p.clip_scale) {
                const float4* s = reinterpret_cast<const float4*>(p.clip_scale + g * D + at_d + 8 * i);
                const float4 a = s[0], b = s[1];
                kx[i][0] *= a.x; kx[i][1] *= a.y; kx[i][2] *= a.z; kx[i][3] *= a.w;
                kx[i][4] *= b.x; kx[i][5] *= b.y; kx[i][6] *= b.z; kx[i][7] *= b.w;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(kx[i][e], kx[i][e], ss);
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(peers, ss, o);
        const float n = sqrtf(ss);
        const float c = (n > p.thr ? p.thr / n : 1.f) * tau;
#pragma unroll
        for (int i = 0; i < PER / 8; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) kx[i][e] *= c;
            ku[i] = pack8_bf16(kx[i]);  // the clip's result is BF16, as inkling_l2clip_fwd's is
        }
    }
    if (slot < 0 || slot >= p.num_slots) return;
    const int page = p.page.index(int(slot));  // slots are below 2^31
    const int64_t at = int64_t(page) * p.page_stride + int64_t(int(slot) - page * p.page.size) * p.token_stride +
                       int64_t(g) * p.head_stride + at_d;
    if constexpr (E4M3) {
        uint2 kc[2], vc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x[8];
            unpack8(ku[i], x);
            kc[i] = pack8_e4m3(x, ks);
            unpack8(vu[i], x);
            vc[i] = pack8_e4m3(x, vs);
        }
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.k_cache) + at) = make_uint4(kc[0].x, kc[0].y, kc[1].x, kc[1].y);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.v_cache) + at) = make_uint4(vc[0].x, vc[0].y, vc[1].x, vc[1].y);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.k_cache) + at) = ku[0];
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v_cache) + at) = vu[0];
    }
}

template <int D>
cudaError_t launch_append(const AppendParams& p, bool e4m3, bool clip, cudaStream_t st) {
    const unsigned rpb = kAppendThreads / (D / (e4m3 ? kPerLane<true> : kPerLane<false>));
    const unsigned blocks = (p.rows + rpb - 1) / rpb;
    const auto kernel = e4m3 ? (clip ? append_kernel<D, true, true> : append_kernel<D, true, false>)
                             : (clip ? append_kernel<D, false, true> : append_kernel<D, false, false>);
    return launch_early(kernel, dim3(blocks), kAppendThreads, 0, st, p);
}

inkling_status status_of(cudaError_t e) {
    return ira::note_cuda_error(e) == cudaSuccess ? INKLING_OK : INKLING_ERR_CUDA;
}

}  // namespace

namespace ira {

inkling_status check_cache(const inkling_kv_cache_desc* c, CacheLayout* out) {
    if (!c) return INKLING_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->page_size <= 0 || c->heads_kv <= 0) return INKLING_ERR_INVALID_ARG;
    if (c->dtype != INKLING_KV_BF16 && c->dtype != INKLING_KV_E4M3) return INKLING_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return INKLING_ERR_UNSUPPORTED;
    if (c->num_pages > 0x7fffffff || c->page_size >= (int64_t(1) << 30) || c->heads_kv >= 65536 ||
        c->num_pages * c->page_size > (int64_t(1) << 31))
        return INKLING_ERR_UNSUPPORTED;
    const int64_t unit = c->dtype == INKLING_KV_BF16 ? 8 : 16;
    const int64_t extent[3] = {c->num_pages, c->page_size, c->heads_kv};
    const int64_t stride[3] = {c->page_stride, c->token_stride, c->head_stride};
    int64_t* to[3] = {&out->page_stride, &out->token_stride, &out->head_stride};
    for (int i = 0; i < 3; ++i) {
        *to[i] = 0;
        if (extent[i] == 1) continue;
        if (stride[i] < c->head_dim || stride[i] % unit != 0) return INKLING_ERR_INVALID_ARG;
        if (stride[i] > (int64_t(1) << 60) / extent[i]) return INKLING_ERR_UNSUPPORTED;
        *to[i] = stride[i];
    }
    out->e4m3 = c->dtype == INKLING_KV_E4M3;
    return INKLING_OK;
}

}  // namespace ira

extern "C" {

inkling_status inkling_kv_plan(const inkling_kv_plan_dims* dims, const int32_t* old_lens, const int32_t* new_lens,
                               int32_t* block_table, int32_t* free_pages, const int32_t* free_count, int32_t* lens,
                               int32_t* query_start, int64_t* slots, int32_t* positions, int32_t* info,
                               void* stream) {
    NvtxRange nvtx_range("inkling_kv_plan");
    const inkling_status s = check_plan(dims);
    if (s != INKLING_OK) return s;
    const size_t N = size_t(dims->requests), T = size_t(dims->max_tokens);
    if (!free_pages || !free_count || !query_start || !info) return INKLING_ERR_INVALID_ARG;
    if (N && (!old_lens || !new_lens || !block_table || !lens)) return INKLING_ERR_INVALID_ARG;
    if (T && (!slots || !positions)) return INKLING_ERR_INVALID_ARG;
    for (const void* q : {static_cast<const void*>(old_lens), static_cast<const void*>(new_lens),
                          static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_count), static_cast<const void*>(lens),
                          static_cast<const void*>(query_start), static_cast<const void*>(positions),
                          static_cast<const void*>(info)})
        if (!aligned(q, 4)) return INKLING_ERR_INVALID_ARG;
    if (!aligned(slots, 8)) return INKLING_ERR_INVALID_ARG;
    // what is written may be read or written nowhere else: the blocks do not wait for each other
    constexpr int kWritten = 7, kBuffers = 10;
    const struct { const void* p; size_t n; } buffers[kBuffers] = {
        {block_table, N * size_t(dims->max_pages) * 4}, {free_pages, size_t(dims->num_pages) * 4}, {lens, N * 4},
        {query_start, (N + 1) * 4}, {slots, T * 8}, {positions, T * 4}, {info, 16},
        {old_lens, N * 4}, {new_lens, N * 4}, {free_count, 4}};
    for (int i = 0; i < kWritten; ++i)
        for (int j = i + 1; j < kBuffers; ++j)
            if (overlap(buffers[i].p, buffers[i].n, buffers[j].p, buffers[j].n)) return INKLING_ERR_INVALID_ARG;

    PlanParams p{int(N), int(dims->max_pages), int(dims->num_pages), int(T), PageDivisor(dims->page_size),
                 old_lens, new_lens, block_table, free_pages, free_count, lens, query_start, slots, positions, info};
    const size_t smem = (N + 1) * 12;
    if (smem + kPlanStatic > 48 * 1024) {  // what a launch gets without asking holds both
        // always to the largest batch's size: a thread that set its own would take the limit from
        // under another one's launch
        const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   int((kPlanMaxRequests + 1) * 12));
        if (e != cudaSuccess) return status_of(e);
    }
    // At most one block per SM of a B200: more would only repeat the prefix sums. The pages taken
    // and returned are not known here and not counted: few requests that give back very many are
    // rounds of the loop on few blocks (16,384 pages of 8 requests 12 us, 262,144 of 8 143 us).
    const size_t want = (T + 2 * N + 1 + kPlanThreads - 1) / kPlanThreads;
    return status_of(launch_early(plan_kernel, dim3(unsigned(want < 148 ? want : 148)), kPlanThreads, smem,
                                  static_cast<cudaStream_t>(stream), p));
}

inkling_status inkling_kv_append(const inkling_kv_cache_desc* cache, const inkling_kv_append_dims* dims,
                                 const uint16_t* k, const uint16_t* v, const int64_t* slots, const float* k_scale,
                                 const float* v_scale, const float* clip_scale, const float* tau, void* k_cache,
                                 void* v_cache, void* stream) {
    NvtxRange nvtx_range("inkling_kv_append");
    CacheLayout lay;
    const inkling_status s = check_cache(cache, &lay);
    if (s != INKLING_OK) return s;
    if (!dims || dims->tokens < 0) return INKLING_ERR_INVALID_ARG;
    const int64_t T = dims->tokens, H = cache->heads_kv, HD = H * cache->head_dim;
    if (T > 1 && (dims->k_row < HD || dims->v_row < HD)) return INKLING_ERR_INVALID_ARG;
    if (dims->k_row % 8 != 0 || dims->v_row % 8 != 0) return INKLING_ERR_INVALID_ARG;
    if (dims->clip_k ? !(dims->threshold >= 0.0) : (clip_scale || tau)) return INKLING_ERR_INVALID_ARG;
    if (lay.e4m3 != (k_scale != nullptr) || lay.e4m3 != (v_scale != nullptr)) return INKLING_ERR_INVALID_ARG;
    if (T >= (int64_t(1) << 31) || T * H >= (int64_t(1) << 31)) return INKLING_ERR_UNSUPPORTED;
    if (T > 1 && (dims->k_row > (int64_t(1) << 60) / T || dims->v_row > (int64_t(1) << 60) / T))
        return INKLING_ERR_UNSUPPORTED;
    if (T == 0) return INKLING_OK;
    if (!k || !v || !slots || !k_cache || !v_cache || k_cache == v_cache) return INKLING_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(clip_scale, 16) || !aligned(slots, 8) || !aligned(tau, 4) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4))
        return INKLING_ERR_INVALID_ARG;
    AppendParams p{unsigned(T * H), PageDivisor(H), PageDivisor(cache->page_size), cache->num_pages * cache->page_size,
                   lay.page_stride, lay.token_stride, lay.head_stride, T > 1 ? dims->k_row : 0,
                   T > 1 ? dims->v_row : 0, float(dims->threshold), k, v, slots, k_scale, v_scale, clip_scale, tau,
                   k_cache, v_cache};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return status_of(cache->head_dim == 128 ? launch_append<128>(p, lay.e4m3, dims->clip_k != 0, st)
                                            : launch_append<64>(p, lay.e4m3, dims->clip_k != 0, st));
}

}  // extern "C"
