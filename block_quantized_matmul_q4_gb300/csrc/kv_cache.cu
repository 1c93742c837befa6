// kv_cache.cu -- the paged 8-bit cache of keys and values: append (rotation,
// block scale, codes) and read (codes back to values).
//
// A block is one page of one head. Its scale is a running maximum, so a block
// that grows re-rounds the codes that it holds: q' = round(q d_old / d). One
// CTA owns a block for the whole call, which makes the maximum, the re-rounding
// and the new codes one pass: the new values (at most page_tokens * head_dim,
// eight pairs' worth of registers for each thread) are read from memory once,
// rotated, reduced to their largest magnitude and written as codes. Both
// kernels are bound by memory traffic for prompts and by the chain of
// dependent loads (row offsets, page id, scale) for a decode step.
#include "serving.cuh"

namespace qmm {
namespace serving {
namespace {

constexpr int kItems = 8;     // items of eight elements that a thread holds
constexpr int kThreadsMax = 512;
static_assert(kThreadsMax * kItems * 8 >= kPageMax * kHeadDimMax, "a block fits its CTA's registers");

__device__ __forceinline__ int code_of(float x, float inv) { return q8_code(x, inv); }
__device__ __forceinline__ uint32_t pack_codes(float4 v, float inv) {
    const uint32_t lo = __byte_perm(code_of(v.x, inv), code_of(v.y, inv), 0x0040);
    const uint32_t hi = __byte_perm(code_of(v.z, inv), code_of(v.w, inv), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
// The largest |x| so far as bits: infinities and NaN order above every number.
__device__ __forceinline__ uint32_t max_bits(uint32_t m, float4 v) {
    m = max(m, __float_as_uint(v.x) & 0x7FFFFFFFu);
    m = max(m, __float_as_uint(v.y) & 0x7FFFFFFFu);
    m = max(m, __float_as_uint(v.z) & 0x7FFFFFFFu);
    return max(m, __float_as_uint(v.w) & 0x7FFFFFFFu);
}

// grid: (units, heads, keys or values). Unit = one page that a sequence
// appends to.
template <int FT>
__global__ void __launch_bounds__(kThreadsMax)
    kv_append_kernel(const Cache c, const Batch g, const Rope rope, const Rows K, const Rows V) {
    pdl_launch_dependents();
    pdl_wait();
    const int P = c.page, D = c.dim;
    const Unit u = find_unit(blockIdx.x, g.batch, [&](int b) {
        const Seq s = seq_at(g, b, P);
        return s.n > 0 ? (s.len - 1) / P - (s.len - s.n) / P + 1 : 0;
    });
    if (u.b < 0) return;
    const Seq s = seq_at(g, u.b, P);
    const int start = s.len - s.n;        // position of the first new token
    const int pg = start / P + u.i;       // page of the sequence
    const int s0 = max(start - pg * P, 0), s1 = min(P, s.len - pg * P);  // its new slots
    const int id = page_at(g, u.b, pg);
    if (id < 0) return;
    const int h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const int64_t block = (int64_t)id * c.heads + h;
    int8_t *codes = (is_v ? c.v : c.k) + block * P * D;
    float *scale = (is_v ? c.vs : c.ks) + block;
    const float d_old = s0 > 0 ? *scale : 0.0f;

    // the block's new values, rotated
    const Rows X = is_v ? V : K;
    const Rope r = is_v ? Rope{nullptr, 0, 0} : rope;
    const int per_row = D / 8, items = (s1 - s0) * per_row;
    float4 a[kItems], b[kItems];
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i < items) {
            const int row = i / per_row, j = i - row * per_row;
            const int2 q = quad_at(r, j);
            const int64_t pos = (int64_t)pg * P + s0 + row;
            const int64_t at = (s.row0 + (pos - start)) * X.stride + (int64_t)h * D;
            a[k] = load4<FT>(X.p, at + q.x);
            b[k] = load4<FT>(X.p, at + q.y);
            rotate_item(r, j, pos, a[k], b[k]);
            most = max_bits(max_bits(most, a[k]), b[k]);
        }
    }
    __shared__ uint32_t warp_most[kThreadsMax / 32];
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) warp_most[threadIdx.x >> 5] = most;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 32; ++w) most = max(most, warp_most[w]);

    const float inf = __int_as_float(0x7F800000);
    float d = most >= 0x7F800000u ? inf : __fdiv_rn(__uint_as_float(most), 127.0f);
    if (d < 1.17549435e-38f) d = 0.0f;  // 1 / d would overflow
    const bool grew = d > d_old;
    if (!grew) d = d_old;
    const bool plain = d > 0.0f && d < inf;
    const float inv = plain ? __fdiv_rn(1.0f, d) : 0.0f;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i < items) {
            const int row = i / per_row, j = i - row * per_row;
            const int2 q = quad_at(r, j);
            int8_t *to = codes + (s0 + row) * D;
            *reinterpret_cast<uint32_t *>(to + q.x) = plain ? pack_codes(a[k], inv) : 0u;
            *reinterpret_cast<uint32_t *>(to + q.y) = plain ? pack_codes(b[k], inv) : 0u;
        }
    }
    if (grew && d_old > 0.0f) {  // the block's other codes, at the new scale
        const float ratio = plain ? __fdiv_rn(d_old, d) : 0.0f;
        uint32_t *kept = reinterpret_cast<uint32_t *>(codes);
        const int words = D / 4, gap = (s1 - s0) * words;
        for (int j = threadIdx.x; j < P * words - gap; j += blockDim.x) {
            const int i = j < s0 * words ? j : j + gap;
            const uint32_t w = kept[i];
            kept[i] = pack_codes(make_float4((float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16),
                                             (float)(int8_t)(w >> 24)), ratio);
        }
    }
    if (threadIdx.x == 0) *scale = d;
}

// grid: (pages, heads, keys or values); each thread 16 codes at a time.
template <int FT>
__global__ void __launch_bounds__(256)
    kv_read_kernel(const Cache c, const int32_t *pages, int64_t num_pages, void *K, void *V, unsigned *err) {
    pdl_launch_dependents();
    pdl_wait();
    const int id = pages[blockIdx.x];
    if (id < 0 || id >= num_pages) {
        if (threadIdx.x == 0) atomicOr(err, kDevErrRange);
        return;
    }
    const int n = c.page * c.dim;
    const bool is_v = blockIdx.z != 0;
    const int64_t block = (int64_t)id * c.heads + blockIdx.y;
    const int8_t *codes = (is_v ? c.v : c.k) + block * n;
    const float d = (is_v ? c.vs : c.ks)[block];
    void *out = is_v ? V : K;
    const int64_t to = ((int64_t)blockIdx.x * c.heads + blockIdx.y) * n;
    for (int i = threadIdx.x; i < n / 16; i += blockDim.x) {
        const uint4 u = reinterpret_cast<const uint4 *>(codes)[i];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            store4<FT>(out, to + 16 * i + 4 * k,
                       make_float4(d * (float)(int8_t)w[k], d * (float)(int8_t)(w[k] >> 8),
                                   d * (float)(int8_t)(w[k] >> 16), d * (float)(int8_t)(w[k] >> 24)));
    }
}

}  // namespace

cudaError_t launch_kv_append(const Cache &c, const Batch &g, const Rope &r, int ft, Rows K, Rows V, cudaStream_t s) {
    // Pages touched: n rows touch at most (n - 2) / page + 2 pages, one row one.
    const int64_t seqs = g.T < g.batch ? g.T : g.batch;
    const int64_t units = g.T / c.page + 2 * seqs < g.T ? g.T / c.page + 2 * seqs : g.T;
    int threads = c.page * c.dim / (8 * kItems);
    threads = threads < 64 ? 64 : (threads + 31) / 32 * 32;
    const dim3 grid((unsigned)units, (unsigned)c.heads, 2);
    auto kernel = ft == QMM_F32 ? kv_append_kernel<QMM_F32> : ft == QMM_F16 ? kv_append_kernel<QMM_F16> : kv_append_kernel<QMM_BF16>;
    return launch(kernel, grid, threads, 0, s, c, g, r, K, V);
}

cudaError_t launch_kv_read(const Cache &c, const int32_t *pages, int64_t n, int64_t num_pages, int ft, void *K, void *V,
                           unsigned *err, cudaStream_t s) {
    const dim3 grid((unsigned)n, (unsigned)c.heads, 2);
    auto kernel = ft == QMM_F32 ? kv_read_kernel<QMM_F32> : ft == QMM_F16 ? kv_read_kernel<QMM_F16> : kv_read_kernel<QMM_BF16>;
    return launch(kernel, grid, 128, 0, s, c, pages, num_pages, K, V, err);
}

}  // namespace serving
}  // namespace qmm
