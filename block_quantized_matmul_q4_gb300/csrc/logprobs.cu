// logprobs.cu -- log probabilities of given tokens, entropy and the most
// likely alternatives, from one pass over the logits.
//
// With d = (x - m) log2 e for any reference m:  l = sum 2^d  and  t = sum 2^d d
// give  lse = m + ln 2 log2 l  and  entropy = (log2 l - t / l) ln 2;  sums with
// references m_c join with d_c = (m_c - m) log2 e as  l = sum 2^d_c l_c,  t =
// sum 2^d_c (t_c + d_c l_c). (The difference is taken before the product:
// logits masked with the type's lowest value would overflow it.)  A CTA holds a chunk of a row in
// registers, so the maximum comes before the exponentials without a second
// read; a row of several chunks is joined by a second kernel.
#include "serving.cuh"

namespace qmm {
namespace serving {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896f;
constexpr int kTopMax = 32;
constexpr int kFoundMax = 256;  // one for each thread: candidates rank themselves
static_assert(kFoundMax <= kThreads, "a thread for each candidate");
constexpr int64_t kVocabMax = (int64_t)1 << 20;
// Elements of a chunk for each thread: 64, or 16 where that leaves SMs idle
// (see chunk_elems).
constexpr int kEltsLarge = 64, kEltsSmall = 16;
constexpr int kListsMax = 96;  // chunks of a row: kVocabMax / (256 * 64) and one more, or kSmallChunksMax
constexpr int kSmallChunksMax = 64;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Logits in falling order, equal ones by rising index, as falling 64-bit keys.
// No element: 0. NaN above +inf; -0 equals 0.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    const uint32_t o = x != x ? 0xFFFFFFFFu : (u & 0x80000000u ? ~u : u | 0x80000000u);
    return (uint64_t)o << 32 | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ int key_index(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The warp's values in falling order, the largest in lane 0 (bitonic).
__device__ __forceinline__ float warp_sort_falling(float v, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k *= 2)
#pragma unroll
        for (int j = k / 2; j; j /= 2) {
            const float o = __shfl_xor_sync(0xffffffffu, v, j);
            // the lower lane of a falling run keeps the larger value
            v = ((lane & j) == 0) == ((lane & k) == 0) ? fmaxf(v, o) : fminf(v, o);
        }
    return v;
}

struct Stats {
    float m, l, t;
};

template <int FT>
__device__ __forceinline__ float load_one(const void *p, int64_t i) {
    if (FT == QMM_F32) return static_cast<const float *>(p)[i];
    const uint16_t u = static_cast<const uint16_t *>(p)[i];
    if (FT == QMM_F16) return __half2float(__ushort_as_half(u));
    return __uint_as_float((uint32_t)u << 16);
}

// The outputs of a row from its joined sums and its `top` keys in shared
// memory, by the whole CTA.
template <int FT>
__device__ __forceinline__ void finish_row(const Logprobs &a, int64_t row, Stats s, const uint64_t *keys) {
    constexpr float kLn2 = 0.693147180559945f;
    const float inf = __int_as_float(0x7F800000);
    const bool none = s.l == 0.0f;  // every logit is -inf
    const float log2l = log2f(s.l);
    const float lse = none ? -inf : fmaf(log2l, kLn2, s.m);
    // (x - m) - log l, not x - lse: the same number, with one rounding less
    // where |m| is large
    auto logp = [&](float x) { return none ? -inf : fmaf(log2l, -kLn2, x - s.m); };
    if (threadIdx.x == 0) {
        if (a.lse) a.lse[row] = lse;
        if (a.entropy) a.entropy[row] = none ? 0.0f : (log2l - s.t / s.l) * kLn2;
    }
    if (a.given_logp)
        for (int g = threadIdx.x; g < a.G; g += blockDim.x) {
            const int id = a.given[row * a.G + g];
            float v = __int_as_float(0x7FC00000);
            if (id >= 0 && id < a.V) v = logp(load_one<FT>(a.X, row * a.stride + id));
            a.given_logp[row * a.G + g] = v;
        }
    for (int k = threadIdx.x; k < a.top; k += blockDim.x) {
        a.top_ids[row * a.top + k] = key_index(keys[k]);
        a.top_logp[row * a.top + k] = logp(key_value(keys[k]));
    }
}

// Pairs of fp32 values: one instruction for two.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// A chunk of a row: `vecs` 16-byte vectors for each thread, vector i of thread
// j at elements first + (i * kThreads + j) * (16 / element size) and on, those
// of them that are in 0 .. V - 1.
struct Chunk {
    const char *row;
    int64_t first, V;
    int vecs;
};

// The chunk's `n` largest keys in falling order by rounds of a CTA-wide
// maximum, read from memory each time: for chunks with many equal logits or a
// NaN, which largest_keys does not take.
template <int FT>
__device__ __noinline__ void largest_keys_by_rounds(const Chunk c, int n, uint64_t *top, uint64_t (*best_of)[kThreads / 32]) {
    constexpr int kVec = FT == QMM_F32 ? 4 : 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t mine = 0, last = ~0ull;
    for (int k = 0; k < n; ++k) {
        if (k == 0 || mine == last) {  // this thread's largest key below the last one taken
            mine = 0;
            for (int i = 0; i < c.vecs; ++i)
                for (int j = 0; j < kVec; ++j) {
                    const int64_t e = c.first + ((int64_t)i * kThreads + threadIdx.x) * kVec + j;
                    const uint64_t key = e >= 0 && e < c.V ? key_of(load_one<FT>(c.row, e), (uint32_t)e) : 0;
                    if (key < last && key > mine) mine = key;
                }
        }
        const uint64_t w = warp_max_key(mine);
        if (lane == 0) best_of[k & 1][warp] = w;
        __syncthreads();
        last = 0;
        for (int i = 0; i < kThreads / 32; ++i) last = best_of[k & 1][i] > last ? best_of[k & 1][i] : last;
        if (threadIdx.x == 0) top[k] = last;
    }
    __syncthreads();
}

// The chunk's `n` largest keys in falling order; most: this thread's largest
// element. The n-th largest of the threads' maxima, tau, bounds the n-th
// largest element from below, so the elements >= tau (little more than n of
// them) hold the answer. Each warp sorts its maxima, every thread ranks its
// one among all by binary searches, the warps read the elements of the
// threads that reach tau once more, and the elements found rank themselves by
// counting. False where more are found than fit.
template <int FT>
__device__ __forceinline__ bool largest_keys(const Chunk c, int n, float most, uint64_t *top) {
    constexpr int kVec = FT == QMM_F32 ? 4 : 8;
    __shared__ float maxima[kThreads / 32][32];
    __shared__ float tau_at;
    __shared__ int threads, count;
    __shared__ int16_t reach[kThreads];
    __shared__ uint64_t found[kFoundMax];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float sorted = warp_sort_falling(most, lane);
    maxima[warp][lane] = sorted;
    if (threadIdx.x == 0) threads = count = 0;
    if ((int)threadIdx.x < n) top[threadIdx.x] = 0;
    __syncthreads();
    int rank = lane;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        // warp w's maxima that come before this one (equal ones: by warp)
        int before = 0;
#pragma unroll
        for (int step = 16; step; step /= 2) {
            const float v = maxima[w][before + step - 1];
            before += v > sorted || (v == sorted && w < warp) ? step : 0;
        }
        const float v = maxima[w][before];
        before += v > sorted || (v == sorted && w < warp) ? 1 : 0;
        rank += w == warp ? 0 : before;
    }
    if (rank == n - 1) tau_at = sorted;
    __syncthreads();
    const float tau = tau_at;
    if (most >= tau) reach[atomicAdd(&threads, 1)] = (int16_t)threadIdx.x;
    __syncthreads();
    for (int t = warp; t < threads; t += kThreads / 32)
        for (int i = lane; i < c.vecs * kVec; i += 32) {
            const int64_t e = c.first + ((int64_t)(i / kVec) * kThreads + reach[t]) * kVec + i % kVec;
            if (e < 0 || e >= c.V) continue;
            const float x = load_one<FT>(c.row, e);
            if (x >= tau) {
                const int at = atomicAdd(&count, 1);
                if (at < kFoundMax) found[at] = key_of(x, (uint32_t)e);
            }
        }
    __syncthreads();
    const int all = count;
    if (all > kFoundMax) return false;
    if ((int)threadIdx.x < all) {
        const uint64_t key = found[threadIdx.x];
        int before = 0;
        for (int i = 0; i < all; ++i) before += found[i] > key;
        if (before < n) top[before] = key;
    }
    __syncthreads();
    return true;
}

// grid: rows x chunks. stats [row][chunk] and keys [row][chunk][top] where a
// row has several chunks.
template <int FT, int ELTS>
__global__ void __launch_bounds__(kThreads, 3) logprobs_chunk_kernel(const Logprobs a, int chunks, Stats *stats, uint64_t *keys) {
    constexpr int kVec = FT == QMM_F32 ? 4 : 8;
    constexpr int kVecs = ELTS / kVec;
    __shared__ float red[3][kThreads / 32];
    __shared__ uint64_t best_of[2][kThreads / 32];
    __shared__ uint64_t top[kTopMax];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x / chunks;
    const int chunk = (int)(blockIdx.x - row * chunks);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float inf = __int_as_float(0x7F800000);

    // the chunk as 16-byte vectors of the row's aligned addresses; vectors
    // that the row's ends cut are read element by element
    constexpr int kSize = FT == QMM_F32 ? 4 : 2;
    Chunk c;
    c.row = static_cast<const char *>(a.X) + row * a.stride * kSize;
    c.V = a.V;
    c.first = (int64_t)chunk * kVecs * kThreads * kVec - (int)((uintptr_t)c.row % 16) / kSize;
    const int64_t left = (a.V - c.first + kThreads * kVec - 1) / (kThreads * kVec);
    c.vecs = left < kVecs ? (int)left : kVecs;  // the last chunk may hold few
    float x[ELTS];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t e = c.first + ((int64_t)i * kThreads + threadIdx.x) * kVec;
        float *v = x + i * kVec;
        if (i < c.vecs && e >= 0 && e + kVec <= a.V) {
            const uint4 u = ld128(c.row + e * kSize);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (FT == QMM_F32) {
                    v[k] = __uint_as_float(w[k]);
                } else if (FT == QMM_F16) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                    v[(2 * k) % kVec] = f.x;
                    v[(2 * k + 1) % kVec] = f.y;
                } else {
                    v[(2 * k) % kVec] = __uint_as_float(w[k] << 16);
                    v[(2 * k + 1) % kVec] = __uint_as_float(w[k] & 0xFFFF0000u);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[k] = e + k >= 0 && e + k < a.V ? load_one<FT>(c.row, e + k) : -inf;
        }
    }
    float mine = -inf;
#pragma unroll
    for (int i = 0; i < ELTS; ++i) mine = fmaxf(mine, x[i]);

    // the chunk's sums
    Stats s;
    float most = mine;
#pragma unroll
    for (int d = 16; d; d /= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    if (lane == 0) red[0][warp] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) most = fmaxf(most, red[0][w]);
    s.m = most == -inf ? 0.0f : most;
    uint64_t l2 = pair(0.0f, 0.0f), t2 = l2;
    const uint64_t minus = pair(-s.m, -s.m), log2e = pair(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        if (i < c.vecs)
#pragma unroll
            for (int k = 0; k < kVec; k += 2) {
                const uint64_t d = mul2(add2(pair(x[i * kVec + k], x[i * kVec + k + 1]), minus), log2e);
                const float2 f = unpair(d);
                const uint64_t e = pair(ex2(f.x), ex2(f.y));
                l2 = add2(l2, e);
                t2 = fma2(e, pair(fmaxf(f.x, -1000.0f), fmaxf(f.y, -1000.0f)), t2);  // 0, not 0 * -inf, where x = -inf
            }
    s.l = unpair(l2).x + unpair(l2).y;
    s.t = unpair(t2).x + unpair(t2).y;
#pragma unroll
    for (int d = 16; d; d /= 2) {
        s.l += __shfl_xor_sync(0xffffffffu, s.l, d);
        s.t += __shfl_xor_sync(0xffffffffu, s.t, d);
    }
    if (lane == 0) {
        red[1][warp] = s.l;
        red[2][warp] = s.t;
    }
    __syncthreads();
    s.l = s.t = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        s.l += red[1][w];
        s.t += red[2][w];
    }

    // a NaN, which the maxima pass over, shows in the sum
    if (a.top && (s.l != s.l || !largest_keys<FT>(c, a.top, mine, top))) largest_keys_by_rounds<FT>(c, a.top, top, best_of);
    if (chunks == 1) {
        finish_row<FT>(a, row, s, top);
        return;
    }
    if (threadIdx.x == 0) stats[blockIdx.x] = s;
    if ((int)threadIdx.x < a.top) keys[(int64_t)blockIdx.x * a.top + threadIdx.x] = top[threadIdx.x];
}

// One CTA joins a row's chunks: the sums, then the first `top` of the chunks'
// falling lists by rounds of a maximum over the lists' heads.
template <int FT>
__global__ void __launch_bounds__(64) logprobs_join_kernel(const Logprobs a, int chunks, const Stats *stats, const uint64_t *keys) {
    __shared__ uint64_t list[kListsMax * kTopMax];
    __shared__ uint64_t top[kTopMax];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < chunks * a.top; i += blockDim.x) list[i] = keys[row * chunks * a.top + i];
    const float inf = __int_as_float(0x7F800000);
    Stats s = {-inf, 0.0f, 0.0f};
    for (int c = lane; c < chunks; c += 32) {
        const Stats p = stats[row * chunks + c];
        if (p.l != 0.0f) s.m = fmaxf(s.m, p.m);
    }
#pragma unroll
    for (int d = 16; d; d /= 2) s.m = fmaxf(s.m, __shfl_xor_sync(0xffffffffu, s.m, d));
    for (int c = lane; c < chunks; c += 32) {
        const Stats p = stats[row * chunks + c];
        if (p.l != 0.0f) {
            const float d = (p.m - s.m) * kLog2e, f = ex2(d);
            s.l += f * p.l;
            s.t = fmaf(f, p.t + fmaxf(d, -1000.0f) * p.l, s.t);
        }
    }
#pragma unroll
    for (int d = 16; d; d /= 2) {
        s.l += __shfl_xor_sync(0xffffffffu, s.l, d);
        s.t += __shfl_xor_sync(0xffffffffu, s.t, d);
    }
    __syncthreads();
    if (threadIdx.x < 32 && a.top) {
        constexpr int kMine = kListsMax / 32;
        uint64_t head[kMine];
        int at[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            at[i] = 0;
            head[i] = lane + 32 * i < chunks ? list[(lane + 32 * i) * a.top] : 0;
        }
        for (int k = 0; k < a.top; ++k) {
            uint64_t mine = 0;
#pragma unroll
            for (int i = 0; i < kMine; ++i) mine = head[i] > mine ? head[i] : mine;
            const uint64_t best = warp_max_key(mine);
            if (lane == 0) top[k] = best;
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                if (head[i] == best && best) {
                    ++at[i];
                    head[i] = at[i] < a.top ? list[(lane + 32 * i) * a.top + at[i]] : 0;
                }
        }
    }
    __syncthreads();
    finish_row<FT>(a, row, s, top);
}

// Elements of a chunk and chunks of a row. Small chunks where the large ones
// would not give every SM a CTA, as long as the join can hold their lists.
struct Split {
    int elts, chunks;
};
Split split_row(int64_t M, int64_t V) {
    auto chunks = [&](int elts) { return (int)((V + 7 + kThreads * elts - 1) / (kThreads * elts)); };
    if (M * chunks(kEltsLarge) < kSms && chunks(kEltsSmall) <= kSmallChunksMax) return {kEltsSmall, chunks(kEltsSmall)};
    return {kEltsLarge, chunks(kEltsLarge)};
}
static_assert((kVocabMax + 7) / (kThreads * kEltsLarge) + 1 <= kListsMax && kSmallChunksMax <= kListsMax, "join's lists");

template <int FT>
cudaError_t launch_typed(const Logprobs &a, Split sp, void *ws, cudaStream_t s) {
    Stats *stats = static_cast<Stats *>(ws);
    uint64_t *keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + align_up((size_t)a.M * sp.chunks * sizeof(Stats), 16));
    auto kernel = sp.elts == kEltsLarge ? logprobs_chunk_kernel<FT, kEltsLarge> : logprobs_chunk_kernel<FT, kEltsSmall>;
    const cudaError_t e = launch(kernel, dim3((unsigned)(a.M * sp.chunks)), kThreads, 0, s, a, sp.chunks, stats, keys);
    if (e != cudaSuccess || sp.chunks == 1) return e;
    return launch(logprobs_join_kernel<FT>, dim3((unsigned)a.M), 64, 0, s, a, sp.chunks, (const Stats *)stats, (const uint64_t *)keys);
}

}  // namespace

size_t logprobs_bytes(int64_t M, int64_t V, int top) {
    const Split sp = split_row(M, V);
    if (sp.chunks == 1) return 0;
    return align_up((size_t)M * sp.chunks * sizeof(Stats), 16) + (size_t)M * sp.chunks * top * 8;
}

cudaError_t launch_logprobs(const Logprobs &a, void *ws, cudaStream_t s) {
    const Split sp = split_row(a.M, a.V);
    if (a.ft == QMM_F32) return launch_typed<QMM_F32>(a, sp, ws, s);
    if (a.ft == QMM_F16) return launch_typed<QMM_F16>(a, sp, ws, s);
    return launch_typed<QMM_BF16>(a, sp, ws, s);
}

}  // namespace serving
}  // namespace qmm
