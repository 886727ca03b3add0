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
    int N, P, M, num_pages, T;
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

constexpr int kPlanThreads = 512;

__device__ __forceinline__ int pages_of(int len, int P) { return len > 0 ? (len - 1) / P + 1 : 0; }

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
// give back) and then independent writes: token i, taken page k and returned page i each
// find their request by bisection. Bound by launch and load latency (a few microseconds
// of work), so it is one kernel with no exchange between blocks: every block computes all
// three sums itself (N <= 16384 lengths, from L2 after the first block) into shared memory
// and takes its share of the writes. The stack needs no order between blocks either: a
// page popped in the same call that returned it is read from the block table, so no block
// reads an entry of free_pages or of the table that another one writes.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanParams p) {
    extern __shared__ int s_at[];
    int* s_tok = s_at;               // [N + 1] exclusive prefix sums, totals at [N]
    int* s_need = s_tok + p.N + 1;
    int* s_back = s_need + p.N + 1;
    __shared__ int3 s_warp[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cap = p.M * p.P;
    auto clamped = [&](int len) { return min(max(len, 0), cap); };

    const int chunk = (p.N + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(tid * chunk, p.N), r1 = min(r0 + chunk, p.N);
    int3 sum = make_int3(0, 0, 0);
    for (int r = r0; r < r1; ++r) {
        const int o = clamped(p.old_lens[r]), w = clamped(p.new_lens[r]);
        const int held = pages_of(o, p.P), want = pages_of(w, p.P);
        s_tok[r] = sum.x;
        s_need[r] = sum.y;
        s_back[r] = sum.z;
        sum.x += max(w - o, 0);
        sum.y += max(want - held, 0);
        sum.z += max(held - want, 0);
    }
    int3 inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc.x, d), y = __shfl_up_sync(0xffffffffu, inc.y, d),
                  z = __shfl_up_sync(0xffffffffu, inc.z, d);
        if (lane >= d) {
            inc.x += x;
            inc.y += y;
            inc.z += z;
        }
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int3 ex = make_int3(inc.x - sum.x, inc.y - sum.y, inc.z - sum.z);
    int3 all = make_int3(0, 0, 0);
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const int3 v = s_warp[w];
        if (w < warp) {
            ex.x += v.x;
            ex.y += v.y;
            ex.z += v.z;
        }
        all.x += v.x;
        all.y += v.y;
        all.z += v.z;
    }
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

    const int count = min(max(*p.free_count, 0), p.num_pages);
    // returned pages beyond the stack's room (malformed tables only) are dropped
    const int back = min(all.z, p.num_pages - count);
    const int avail = count + back;
    const int taken = min(all.y, avail);
    const int left = avail - taken;

    // i-th returned page and k-th taken page
    auto returned = [&](int i) {
        const int r = last_at_or_below(s_back, p.N, i);
        const int want = pages_of(clamped(p.new_lens[r]), p.P);
        return p.table[int64_t(r) * p.M + want + (i - s_back[r])];
    };
    auto popped = [&](int k) {
        const int at = avail - 1 - k;
        return at < count ? p.free_pages[at] : returned(at - count);
    };

    const int gid = blockIdx.x * kPlanThreads + tid, stride = gridDim.x * kPlanThreads;
    for (int i = gid; i < p.T; i += stride) {
        int64_t slot = -1;
        int pos = 0;
        if (i < all.x) {
            const int r = last_at_or_below(s_tok, p.N, i);
            const int o = clamped(p.old_lens[r]);
            const int held = pages_of(o, p.P);
            pos = o + (i - s_tok[r]);
            const int idx = pos / p.P;
            int page = -1;
            if (idx < held) {
                page = p.table[int64_t(r) * p.M + idx];
            } else {
                const int k = s_need[r] + (idx - held);
                if (k < taken) page = popped(k);
            }
            if (page >= 0 && page < p.num_pages) slot = int64_t(page) * p.P + (pos - idx * p.P);
        }
        p.slots[i] = slot;
        p.positions[i] = pos;
    }
    for (int k = gid; k < taken; k += stride) {
        const int r = last_at_or_below(s_need, p.N, k);
        const int held = pages_of(clamped(p.old_lens[r]), p.P);
        p.table[int64_t(r) * p.M + held + (k - s_need[r])] = popped(k);
    }
    // returned pages that this call does not pop again
    for (int i = gid; i < back && count + i < left; i += stride) p.free_pages[count + i] = returned(i);
    for (int r = gid; r <= p.N; r += stride) {
        p.query_start[r] = s_tok[r];
        if (r == p.N) break;
        const int o = clamped(p.old_lens[r]), w = clamped(p.new_lens[r]);
        const int64_t given = min(max(taken - s_need[r], 0), s_need[r + 1] - s_need[r]);
        const int64_t room = (pages_of(o, p.P) + given) * p.P;
        p.lens[r] = w <= o ? w : int(room < w ? room : w);
    }
    if (gid == 0) {
        p.info[0] = left;
        p.info[1] = all.x;
        p.info[2] = all.y - taken;
        p.info[3] = taken;
    }
}

inkling_status check_plan(const inkling_kv_plan_dims* d) {
    if (!d) return INKLING_ERR_INVALID_ARG;
    if (d->requests < 0 || d->page_size <= 0 || d->max_pages <= 0 || d->num_pages <= 0 || d->max_tokens < 0)
        return INKLING_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 30;
    if (d->requests > 16384 || d->page_size >= lim || d->max_pages >= lim || d->num_pages > 0x7fffffff ||
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
    unsigned Hkv, P;
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

constexpr int kAppendThreads = 256;

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

// x / scale, saturated and rounded to nearest even. A true division, so that the codes
// are those of the formula at every tie.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// One (token, head) row of k and of v per group of D / 8 lanes, 8 values of each to a
// lane: 16-byte loads, 16-byte (BF16) or 8-byte (e4m3) stores, all rows of a token next
// to each other. A stream of 4 (or 3) bytes per value, bound by HBM: no loop, so that a
// full SM keeps 2048 threads x 32 bytes in flight. The clip's sum of squares is FP32 over
// the group by shuffles.
template <int D, bool E4M3, bool CLIP>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendParams p) {
    constexpr int LPR = D / 8;
    const unsigned row = blockIdx.x * (kAppendThreads / LPR) + threadIdx.x / LPR;
    const int part = threadIdx.x % LPR;
    const unsigned t = row / p.Hkv, g = row - t * p.Hkv;
    const int64_t slot = row < p.rows ? p.slots[t] : -1;
    const bool live = slot >= 0 && slot < p.num_slots;
    uint4 ku = make_uint4(0, 0, 0, 0), vu = ku;
    if (live) {
        ku = __ldcs(reinterpret_cast<const uint4*>(p.k + t * p.k_row + g * D + part * 8));
        vu = __ldcs(reinterpret_cast<const uint4*>(p.v + t * p.v_row + g * D + part * 8));
    }
    float kx[8];
    if constexpr (CLIP) {
        unpack8(ku, kx);
        if (p.clip_scale && live) {
            const float4* s = reinterpret_cast<const float4*>(p.clip_scale + g * D + part * 8);
            const float4 a = s[0], b = s[1];
            kx[0] *= a.x; kx[1] *= a.y; kx[2] *= a.z; kx[3] *= a.w;
            kx[4] *= b.x; kx[5] *= b.y; kx[6] *= b.z; kx[7] *= b.w;
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(kx[i], kx[i], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float n = sqrtf(ss);
        const float c = (n > p.thr ? p.thr / n : 1.f) * (p.tau && live ? p.tau[t] : 1.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) kx[i] *= c;
        ku = pack8_bf16(kx);  // the clip's result is BF16, as inkling_l2clip_fwd's is
    }
    if (!live) return;
    const unsigned page = unsigned(slot) / p.P;  // slots are below 2^32
    const int64_t at = int64_t(page) * p.page_stride + int64_t(unsigned(slot) - page * p.P) * p.token_stride +
                       int64_t(g) * p.head_stride + part * 8;
    if constexpr (E4M3) {
        float vx[8];
        unpack8(ku, kx);
        unpack8(vu, vx);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.k_cache) + at) = pack8_e4m3(kx, p.k_scale[g]);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.v_cache) + at) = pack8_e4m3(vx, p.v_scale[g]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.k_cache) + at) = ku;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v_cache) + at) = vu;
    }
}

template <int D>
void launch_append(const AppendParams& p, bool e4m3, bool clip, cudaStream_t st) {
    constexpr unsigned rpb = kAppendThreads / (D / 8);
    const unsigned blocks = (p.rows + rpb - 1) / rpb;
    if (e4m3 && clip) append_kernel<D, true, true><<<blocks, kAppendThreads, 0, st>>>(p);
    else if (e4m3) append_kernel<D, true, false><<<blocks, kAppendThreads, 0, st>>>(p);
    else if (clip) append_kernel<D, false, true><<<blocks, kAppendThreads, 0, st>>>(p);
    else append_kernel<D, false, false><<<blocks, kAppendThreads, 0, st>>>(p);
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
        c->num_pages * c->page_size > (int64_t(1) << 32))
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
    const struct { const void* p; size_t n; } in[] = {
        {old_lens, N * 4}, {new_lens, N * 4}, {block_table, N * size_t(dims->max_pages) * 4},
        {free_pages, size_t(dims->num_pages) * 4}, {free_count, 4}};
    const struct { const void* p; size_t n; } outs[] = {
        {lens, N * 4}, {query_start, (N + 1) * 4}, {slots, T * 8}, {positions, T * 4}, {info, 16}};
    for (const auto& o : outs)
        for (const auto& i : in)
            if (overlap(o.p, o.n, i.p, i.n)) return INKLING_ERR_INVALID_ARG;
    if (overlap(block_table, N * size_t(dims->max_pages) * 4, free_pages, size_t(dims->num_pages) * 4))
        return INKLING_ERR_INVALID_ARG;

    PlanParams p{int(N), int(dims->page_size), int(dims->max_pages), int(dims->num_pages), int(T),
                 old_lens, new_lens, block_table, free_pages, free_count, lens, query_start, slots, positions, info};
    const size_t smem = (N + 1) * 12;
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return status_of(e);
    }
    // Tokens and table entries are spread over at most one block per SM: more would only
    // repeat the prefix sums.
    const size_t items = T > N + 1 ? T : N + 1;
    const size_t want = (items + kPlanThreads - 1) / kPlanThreads;
    plan_kernel<<<unsigned(want < 148 ? want : 148), kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return status_of(cudaGetLastError());
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
    if (!k || !v || !slots || !k_cache || !v_cache) return INKLING_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(clip_scale, 16) || !aligned(slots, 8) || !aligned(tau, 4) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4))
        return INKLING_ERR_INVALID_ARG;
    AppendParams p{unsigned(T * H), unsigned(H), unsigned(cache->page_size), cache->num_pages * cache->page_size,
                   lay.page_stride, lay.token_stride, lay.head_stride, T > 1 ? dims->k_row : 0,
                   T > 1 ? dims->v_row : 0, float(dims->threshold), k, v, slots, k_scale, v_scale, clip_scale, tau,
                   k_cache, v_cache};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->head_dim == 128) launch_append<128>(p, lay.e4m3, dims->clip_k != 0, st);
    else launch_append<64>(p, lay.e4m3, dims->clip_k != 0, st);
    return status_of(cudaGetLastError());
}

}  // extern "C"
