// Log probabilities of given tokens, the entropy and the top alternatives of rows of logits.
//
//   y = z log2(e) / T,  S = sum 2^(y - M),  W = sum 2^(y - M) (y - M)
//   logp[id] = ln 2 (y_id - M - log2 S),  entropy = ln 2 (log2 S - W / S)
// One pass over the row for all three sums: a thread's reference M is the maximum
// of its first elements, moved only when a later one passes it by more than 2^8,
// so that the loop is loads, one product and sum, one exponential and two sums an
// element.  y is never rounded (it is an operand of a fused product and sum), so any
// reference serves that is near the maximum; rows whose maximum is past 2^20 in y take
// differences of logits first, in a second pass.
//
// Alternatives cost the pass one maximum an element: a thread keeps its largest
// logit and where it met it first.  Order all elements by (logit, then lowest
// index).  Were a thread that holds one of the K best not among the K threads whose
// own best are first in that order, K elements would be before it; so the K best
// lie with these K threads, at or before the K-th of their bests.  Those threads'
// elements are read once more (from L2), and the few at or before that place are
// ranked by counting.
//
// A row is cut among 1 to 8 CTAs of a cluster, which join their parts through
// distributed shared memory in a fixed order: results repeat bit for bit.
#include "internal.h"
#include "tree.h"

namespace dfl {

namespace {

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_UNROLL = 4;       // 16-byte loads in flight per thread
constexpr int LP_CAND = 512;       // candidates ranked at once
constexpr float LP_LAZY = 8.f;     // a thread's reference moves when passed by more (log2)
constexpr float LP_FAR = 1048576.f;  // references stay within: rounded by 2^-5 at most, which a sum takes
constexpr float LP_TINY = -1000.f; // exponents stay above: 2^-1000 is 0 and 0 * -1000 is 0, where 0 * -inf is NaN
constexpr float LN2 = 0.69314718055994531f;

template <typename T>
struct LpVec;
template <>
struct LpVec<float> {
    static constexpr int N = 4;
    static constexpr uint32_t NONE = 0xFF800000u;     // -inf
    static __device__ __forceinline__ void get(const uint4& r, float (&z)[4]) {
        z[0] = __uint_as_float(r.x); z[1] = __uint_as_float(r.y); z[2] = __uint_as_float(r.z); z[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
};
template <>
struct LpVec<__nv_bfloat16> {
    static constexpr int N = 8;
    static constexpr uint32_t NONE = 0xFF80FF80u;
    static __device__ __forceinline__ void get(const uint4& r, float (&z)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) { z[2 * i] = bf16lo(w[i]); z[2 * i + 1] = bf16hi(w[i]); }
    }
    static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ uint4 ldg_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Order of elements: larger logits first, then lower indices.  Not for NaN.
__device__ __forceinline__ uint64_t lp_key(float z, uint32_t i) {
    const uint32_t b = __float_as_uint(z + 0.f);   // -0 as 0
    return (uint64_t)(b >> 31 ? ~b : b | 0x80000000u) << 32 | (0xFFFFFFFFu - i);
}
__device__ __forceinline__ float lp_key_value(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o >> 31 ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint32_t lp_key_index(uint64_t k) { return 0xFFFFFFFFu - (uint32_t)k; }

// Sums of part of a row by the reference m.
struct LpSums {
    float m, s, w;
    __device__ __forceinline__ void move(float mn) {   // to a reference that is no lower
        const float d = m - mn, f = ex2_ftz(d);
        w = f == 0.f ? 0.f : f * fmaf(d, s, w);
        s *= f;
        m = mn;
    }
    __device__ __forceinline__ void join(LpSums o) {
        const float mn = fmaxf(m, o.m);
        move(mn);
        o.move(mn);
        s += o.s;
        w += o.w;
    }
};

struct LpPart {              // what a CTA of a row's cluster leaves for the first of them
    LpSums sum;
    float zmax;
    int top;                 // its best elements, first come first
    uint64_t key[LP_MAX_TOP];
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t a) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(LP_THREADS, 4) token_logprobs_kernel(const LpArgs a, int C, const DevErr err) {
    using Vec = LpVec<T>;
    constexpr int EPV = Vec::N;
    __shared__ LpPart part;
    __shared__ LpSums red[LP_WARPS];
    __shared__ float red_z[LP_WARPS];
    __shared__ float best_z[LP_THREADS];      // threads' largest logits,
    __shared__ uint32_t best_v[LP_THREADS];   // the vectors they were met in first
    __shared__ int hot[LP_MAX_TOP];           // threads with the first of these, in their order
    __shared__ uint64_t cand[LP_CAND];
    __shared__ uint64_t warp_key[LP_WARPS];
    __shared__ int n_cand;
    grid_dep_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / C;
    const int rank = (int)(blockIdx.x - row * C);
    const T* z0 = static_cast<const T*>(a.logits) + row * a.stride;
    // the row as 16-byte vectors: vector v holds elements v EPV - head .. + EPV - 1
    const int head = (int)((reinterpret_cast<uintptr_t>(z0) & 15) / sizeof(T));
    const uint4* vec = reinterpret_cast<const uint4*>(z0 - head);
    const int nv = (head + a.V + EPV - 1) / EPV, whole0 = head > 0, whole1 = (head + a.V) / EPV;
    const int per = (nv + C - 1) / C, v0 = min(nv, rank * per), v1 = min(nv, v0 + per);
    // elements of vector v that belong to the row, the others as -inf
    auto load = [&](int v, float (&z)[EPV]) {
        if (v >= whole0 && v < whole1) { Vec::get(vec[v], z); return; }
        #pragma unroll
        for (int e = 0; e < EPV; ++e) {
            const int i = v * EPV - head + e;
            z[e] = i >= 0 && i < a.V ? Vec::one(z0 + i) : -INFINITY;
        }
    };

    LpSums t{-LP_FAR, 0.f, 0.f};
    float zmax = -INFINITY;
    uint32_t zat = 0xFFFFFFFFu;
    auto add = [&](const float (&z)[EPV], int v) {
        float m4[2] = {z[0], z[1]};
        #pragma unroll
        for (int e = 2; e < EPV; e += 2) { m4[0] = fmaxf(m4[0], z[e]); m4[1] = fmaxf(m4[1], z[e + 1]); }
        const float mx = fmaxf(m4[0], m4[1]);
        if (TOP && (mx > zmax || (mx == zmax && (uint32_t)v < zat))) zat = (uint32_t)v;
        zmax = fmaxf(zmax, mx);
        const float ref = mx * a.c;
        if (ref > t.m + LP_LAZY) t.move(ref);
        #pragma unroll
        for (int e = 0; e < EPV; ++e) {
            const float d = max_nan(fmaf(z[e], a.c, -t.m), LP_TINY), p = ex2_ftz(d);
            t.s += p;
            t.w = fmaf(p, d, t.w);
        }
    };
    const int lo = max(v0, whole0), hi = min(v1, whole1);
    #pragma unroll 1
    for (int v = v0 + tid; v < hi; v += LP_UNROLL * LP_THREADS) {
        uint4 raw[LP_UNROLL];
        #pragma unroll
        for (int u = 0; u < LP_UNROLL; ++u) {
            const int at = v + u * LP_THREADS;
            raw[u] = make_uint4(Vec::NONE, Vec::NONE, Vec::NONE, Vec::NONE);
            if (at >= lo && at < hi) raw[u] = ldg_stream(vec + at);
        }
        #pragma unroll
        for (int u = 0; u < LP_UNROLL; ++u) {
            float z[EPV];
            Vec::get(raw[u], z);
            add(z, v + u * LP_THREADS);
        }
    }
    // the row's ends, where they share a vector with something else
    #pragma unroll 1
    for (int end = 0; end < 2; ++end) {
        const int v = end ? nv - 1 : 0;
        if (v >= v0 && v < v1 && (end ? v >= whole1 && v >= whole0 : v < whole0) && (v - v0) % LP_THREADS == tid) {
            float z[EPV];
            load(v, z);
            add(z, v);
        }
    }

    // ---- sums of the CTA
    if (TOP) { best_z[tid] = zmax; best_v[tid] = zat; }
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        LpSums q;
        q.m = __shfl_xor_sync(0xFFFFFFFFu, t.m, o);
        q.s = __shfl_xor_sync(0xFFFFFFFFu, t.s, o);
        q.w = __shfl_xor_sync(0xFFFFFFFFu, t.w, o);
        t.join(q);
        zmax = fmaxf(zmax, __shfl_xor_sync(0xFFFFFFFFu, zmax, o));
    }
    if (lane == 0) { red[warp] = t; red_z[warp] = zmax; }
    if (tid == 0) n_cand = 0;
    if (TOP && tid < LP_MAX_TOP) hot[tid] = -1;
    __syncthreads();
    t = red[0];
    zmax = red_z[0];
    #pragma unroll 1
    for (int w = 1; w < LP_WARPS; ++w) { t.join(red[w]); zmax = fmaxf(zmax, red_z[w]); }

    // ---- the CTA's best K elements
    if constexpr (TOP) {
        const float bz = best_z[tid];
        const uint32_t bv = best_v[tid];
        int before = 0;
        #pragma unroll 4
        for (int j = 0; j < LP_THREADS; ++j) {
            const float oz = best_z[j];
            before += oz > bz || (oz == bz && best_v[j] < bv);
        }
        if (before < a.K && bz > -INFINITY) hot[before] = tid;
        __syncthreads();
        // the last of them has the place to reach: its first largest element
        int nh = 0;
        while (nh < a.K && hot[nh] >= 0) ++nh;
        uint64_t least = 0;
        if (nh == a.K) {   // (fewer: every element above -inf is a candidate)
            const int th = hot[nh - 1];
            const float oz = best_z[th];
            float z[EPV];
            load((int)best_v[th], z);
            #pragma unroll
            for (int e = EPV - 1; e >= 0; --e)
                if (z[e] == oz) least = lp_key(oz, (uint32_t)((int)best_v[th] * EPV - head + e));
        }
        const int len = (v1 - v0 + LP_THREADS - 1) / LP_THREADS;   // vectors of a thread, at most
        auto each = [&](auto&& f) {
            #pragma unroll 1
            for (int64_t i = tid; i < (int64_t)nh * len; i += LP_THREADS) {
                const int h = (int)(i / len), v = v0 + hot[h] + (int)(i - (int64_t)h * len) * LP_THREADS;
                if (v >= v1) continue;
                float z[EPV];
                load(v, z);
                #pragma unroll
                for (int e = 0; e < EPV; ++e)
                    if (z[e] > -INFINITY) f(lp_key(z[e], (uint32_t)(v * EPV - head + e)));
            }
        };
        each([&](uint64_t key) {
            if (key >= least) {
                const int c = atomicAdd(&n_cand, 1);
                if (c < LP_CAND) cand[c] = key;
            }
        });
        __syncthreads();
        const int nc = n_cand;
        if (nc <= LP_CAND) {
            #pragma unroll 1
            for (int c = tid; c < nc; c += LP_THREADS) {
                const uint64_t key = cand[c];
                int r = 0;
                #pragma unroll 1
                for (int j = 0; j < nc; ++j) r += cand[j] > key;
                if (r < a.K) part.key[r] = key;
            }
            if (tid == 0) part.top = min(nc, a.K);
        } else {   // many before that place, as in a sorted row: one after the other
            uint64_t last = ~0ull;
            int r = 0;
            #pragma unroll 1
            for (; r < a.K; ++r) {
                uint64_t best = 0;
                each([&](uint64_t key) { if (key < last && key > best) best = key; });
                #pragma unroll
                for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
                __syncthreads();
                if (lane == 0) warp_key[warp] = best;
                __syncthreads();
                for (int w = 0; w < LP_WARPS; ++w) best = max(best, warp_key[w]);
                if (best == 0) break;
                if (tid == 0) part.key[r] = best;
                last = best;
            }
            if (tid == 0) part.top = r;
        }
    }
    if (tid == 0) { part.sum = t; part.zmax = zmax; }
    __syncthreads();

    // ---- the row's sums, from the cluster's parts in their order
    const uint32_t base = smem_u32(&part);
    auto word = [&](int r, const void* p) {
        return ld_cluster_u32(mapa_shared(base, (uint32_t)r) + (uint32_t)(static_cast<const uint8_t*>(p) - reinterpret_cast<const uint8_t*>(&part)));
    };
    auto join_all = [&] {
        if (C == 1) return;
        cluster_sync();
        #pragma unroll 1
        for (int r = 0; r < C; ++r) {
            LpSums o{__uint_as_float(word(r, &part.sum.m)), __uint_as_float(word(r, &part.sum.s)), __uint_as_float(word(r, &part.sum.w))};
            const float oz = __uint_as_float(word(r, &part.zmax));
            if (r == 0) { t = o; zmax = oz; }
            else { t.join(o); zmax = fmaxf(zmax, oz); }
        }
    };
    join_all();
    // A row whose largest logit has no such reference: differences first, then products.
    const bool far = fabsf(zmax) < INFINITY && !(fabsf(zmax * a.c) < LP_FAR);
    if (far) {
        if (C > 1) cluster_sync();   // the parts have been read
        t = LpSums{0.f, 0.f, 0.f};
        #pragma unroll 1
        for (int v = v0 + tid; v < v1; v += LP_THREADS) {
            float z[EPV];
            load(v, z);
            #pragma unroll
            for (int e = 0; e < EPV; ++e) {
                const float d = max_nan((z[e] - zmax) * a.c, LP_TINY), p = ex2_ftz(d);
                t.s += p;
                t.w = fmaf(p, d, t.w);
            }
        }
        t.s = warp_sum(t.s);
        t.w = warp_sum(t.w);
        __syncthreads();
        if (lane == 0) red[warp] = t;
        __syncthreads();
        t = red[0];
        for (int w = 1; w < LP_WARPS; ++w) { t.s += red[w].s; t.w += red[w].w; }
        if (tid == 0) part.sum = t;
        __syncthreads();
        join_all();
    }

    if (rank == 0) {
        if (zmax == -INFINITY) t.s = __int_as_float(0x7FFFFFFF);   // every logit is -inf: no distribution
        const float ls = log2f(t.s);
        const double ref = far ? (double)zmax * a.c : (double)t.m;
        auto logp = [&](float z) {
            if (z == -INFINITY) return t.s != t.s ? t.s : -INFINITY;
            return (float)(((double)z * a.c - ref - ls) * 0.69314718055994531);   // (a product may pass fp32's range)
        };
        if (tid < a.M) {
            #pragma unroll 1
            for (int i = tid; i < a.M; i += LP_THREADS) {
                const int64_t at = row * a.M + i;
                const int id = a.ids[at];
                if (DFL_IN_BOUNDS(err.word, at, a.rows * a.M))
                    a.logp[at] = id >= 0 && id < a.V ? logp(Vec::one(z0 + id)) : -INFINITY;
            }
        }
        if (tid == 0 && a.entropy && DFL_IN_BOUNDS(err.word, row, a.rows)) a.entropy[row] = (ls - t.w / t.s) * LN2;
        if constexpr (TOP) {
            auto put = [&](int r, uint64_t key) {
                const int64_t at = row * a.K + r;
                if (!DFL_IN_BOUNDS(err.word, at, a.rows * a.K)) return;
                a.top_ids[at] = key ? (int)lp_key_index(key) : -1;
                a.top_logp[at] = key ? logp(lp_key_value(key)) : -INFINITY;
            };
            if (C == 1) {
                if (tid < a.K) put(tid, tid < part.top ? part.key[tid] : 0);
            } else {   // ranks among the parts' best: at most 8 * 64
                int all = 0;
                #pragma unroll 1
                for (int r = 0; r < C; ++r) {
                    const int n = (int)word(r, &part.top);
                    #pragma unroll 1
                    for (int i = tid; i < n; i += LP_THREADS) cand[all + i] = ld_cluster_u64(mapa_shared(base, (uint32_t)r) +
                        (uint32_t)(reinterpret_cast<const uint8_t*>(&part.key[i]) - reinterpret_cast<const uint8_t*>(&part)));
                    all += n;
                }
                __syncthreads();
                #pragma unroll 1
                for (int c = tid; c < all; c += LP_THREADS) {
                    const uint64_t key = cand[c];
                    int r = 0;
                    #pragma unroll 1
                    for (int j = 0; j < all; ++j) r += cand[j] > key;
                    if (r < a.K) put(r, key);
                }
                if (tid >= all && tid < a.K) put(tid, 0);
            }
        }
    }
    if (C > 1) cluster_sync();   // the parts stay until the first CTA has read them
}

constexpr int LP_SMS = 152, LP_PER_SM = 4, LP_MAX_CLUSTER = 8;

// CTAs of a row: enough to fill the SMs, with some 16 KB of the row for each.
int lp_cluster(int64_t rows, int64_t row_bytes) {
    int C = 1;
    while (C < LP_MAX_CLUSTER && rows * C * 2 <= LP_SMS * LP_PER_SM && row_bytes / (2 * C) >= 16384) C *= 2;
    return C;
}

template <typename K>
dfl_status launch_cluster(K kern, unsigned grid, int C, cudaStream_t st, const LpArgs& a, const DevErr& err) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(LP_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl_on() ? 2 : 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, a, C, err));
}

}  // namespace

dfl_status token_logprobs_run(DeviceCtx* ctx, const LpArgs& a, int dt, cudaStream_t st) {
    ProfScope ps("token_logprobs", st);
    const int C = lp_cluster(a.rows, (int64_t)a.V * (dt == DFL_BF16 ? 2 : 4));
    const DevErr err = dev_err(ctx);
    const unsigned grid = (unsigned)(a.rows * C);
    if (dt == DFL_BF16)
        return a.K > 0 ? launch_cluster(token_logprobs_kernel<__nv_bfloat16, true>, grid, C, st, a, err)
                       : launch_cluster(token_logprobs_kernel<__nv_bfloat16, false>, grid, C, st, a, err);
    return a.K > 0 ? launch_cluster(token_logprobs_kernel<float, true>, grid, C, st, a, err)
                   : launch_cluster(token_logprobs_kernel<float, false>, grid, C, st, a, err);
}

}  // namespace dfl
