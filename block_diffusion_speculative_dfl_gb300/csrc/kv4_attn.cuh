// What the two attention kernels over the 4-bit paged cache share: arguments,
// the line of work units and the sum of partials (kv4_attn.cu says how the
// line is cut).
#pragma once

#include "internal.h"
#include "kv4.cuh"

namespace dfl {

struct KaArgs {
    Kv4Slab slab;
    const int32_t* table;
    const int32_t* len;
    int max_pages;
    int N, B, Hq, G, R;
    int subs;                 // row tiles per K/V head
    int HS;                   // Hkv * subs
    const __nv_bfloat16* Q;   // [N*B][Hq][hd]
    const __nv_bfloat16* Kb;  // [N*B][Hkv][hd]
    const __nv_bfloat16* Vb;
    __nv_bfloat16* O;         // [N*B][Hq][hd]
    float* Opart;             // [2 * grid][rows][hd]
    float2* ml;               // [2 * grid][rows] (maximum in log2 units, sum)
    float scale_log2;         // log2(e) / sqrt(hd)
    float k_pow2, v_pow2, v_inv;   // 2^k_exp, 2^v_exp, 2^-v_exp
};

// The tensor-memory kernel (kv4_attn_tc.cu): rows of its triples, scratch, launch
// (a complete but for Opart and ml; `units` an upper bound on the line).
inline int kv4_attn_tc_rows(int R) { return R <= 64 ? 64 : 128; }
size_t kv4_attn_tc_ws_bytes(int R, int hd);
dfl_status kv4_attn_tc_run(DeviceCtx* ctx, KaArgs a, int hd, int64_t units, void* ws, cudaStream_t st);

namespace {

constexpr int KA_UNIT = 64;        // keys per unit
constexpr float KA_LAZY = 8.f;     // rescale when a maximum grows by more (log2)
constexpr float KA_LIFT = 7.f;     // P is 2^7 above its nominal value

__device__ __forceinline__ int ka_len(const KaArgs& a, int n, const DevErr& err) {
    const int l = a.len[n], cap = a.max_pages * a.slab.page;
    if (l >= 0 && l <= cap) return l;
    record_error(err, DFL_ERR_INVALID_ARG);
    return min(max(l, 0), cap);
}

__device__ __forceinline__ int ka_units(int len) { return (len + KA_UNIT - 1) / KA_UNIT + 1; }

// The line of units and where position x falls on it.
struct KaLine {
    int total, per;     // units in all, per range
    int n, before;      // sequence that holds x, units of the line before it
};

template <int THREADS>
struct KaLineSmem {
    int red[THREADS / 32];
    int n, before;
};

// The line cut into `ranges`; x = at(per, total) is located when 0 <= x < total.
// All threads of the block call.
template <int THREADS, typename At>
__device__ __forceinline__ KaLine ka_locate(const KaArgs& a, int ranges, KaLineSmem<THREADS>& sm, const DevErr& err, At at) {
    const int chunk = (a.N + THREADS - 1) / THREADS;
    const int n0 = min(a.N, (int)threadIdx.x * chunk), n1 = min(a.N, n0 + chunk);
    int sum = 0;
    for (int n = n0; n < n1; ++n) sum += ka_units(ka_len(a, n, err));
    sum *= a.HS;
    KaLine l;
    const int pre = block_exscan<THREADS>(sum, sm.red, &l.total);
    l.per = max(1, (l.total + ranges - 1) / ranges);
    const int x = at(l.per, l.total);
    if (x >= pre && x < pre + sum) {
        int p = pre;
        for (int n = n0; n < n1; ++n) {
            const int w = ka_units(ka_len(a, n, err)) * a.HS;
            if (x < p + w) { sm.n = n; sm.before = p; break; }
            p += w;
        }
    }
    __syncthreads();
    l.n = sm.n;
    l.before = sm.before;
    return l;
}

// A position on the line as (sequence, head and row tile, unit).
struct KaPos {
    int n, hs, u, nu, len;
    __device__ __forceinline__ void next_triple(const KaArgs& a, const DevErr& err) {
        u = 0;
        if (++hs == a.HS) {
            hs = 0;
            if (++n < a.N) { len = ka_len(a, n, err); nu = ka_units(len); }
        }
    }
};

// Adds up the triple that starts in range blockIdx.x and ends past it: partials
// of that range (its second) and of the following ones (their first), in the
// order of the keys.  gridDim.x ranges; blockIdx.y takes rows of KJ_ROWS.
constexpr int KJ_ROWS = 8;
template <int HD, int ROWS>
__global__ void __launch_bounds__(HD / 4 * KJ_ROWS) kv4_attn_join_kernel(const KaArgs a, const DevErr err) {
    constexpr int TPR = HD / 4, THREADS = TPR * KJ_ROWS;
    __shared__ KaLineSmem<THREADS> line_sm;
    grid_dep_begin();
    const KaLine line = ka_locate<THREADS>(a, gridDim.x, line_sm, err, [&](int per, int total) {
        const int64_t end = ((int64_t)blockIdx.x + 1) * per;   // a triple crosses the border before `end`
        return end < total ? (int)end : -1;
    });
    const int64_t endl = ((int64_t)blockIdx.x + 1) * line.per;
    if (endl >= line.total) return;
    const int end = (int)endl;
    const int nu = ka_units(ka_len(a, line.n, err));
    const int hs = (end - line.before) / nu;
    const int p0 = line.before + hs * nu, p1 = p0 + nu;   // the triple holding unit `end`
    if (p0 == end || p0 < end - line.per) return;          // none crosses, or it started before this CTA
    const int first = blockIdx.x, last = (p1 - 1) / line.per;
    const int head = hs / a.subs, row0 = (hs - head * a.subs) * ROWS;
    const int row = blockIdx.y * KJ_ROWS + threadIdx.x / TPR, c = (threadIdx.x % TPR) * 4, r = row0 + row;
    if (row >= ROWS || r >= a.R) return;
    float M = -INFINITY, L = 0.f;
    for (int j = first; j <= last; ++j) M = fmaxf(M, a.ml[(2 * j + (j == first)) * ROWS + row].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    #pragma unroll 4
    for (int j = first; j <= last; ++j) {
        const int64_t at = (int64_t)(2 * j + (j == first)) * ROWS + row;
        const float2 ml = a.ml[at];
        const float4 v = *reinterpret_cast<const float4*>(a.Opart + at * HD + c);
        const float f = ml.x == -INFINITY ? 0.f : ex2_ftz(ml.x - M);
        L += f * ml.y;
        o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
    }
    const float inv = a.v_pow2 / L;
    const int64_t at = ((int64_t)(line.n * a.B + r / a.G) * a.Hq + head * a.G + r % a.G) * HD + c;
    if (DFL_IN_BOUNDS(err.word, at + 3, (int64_t)a.N * a.B * a.Hq * HD))
        *reinterpret_cast<uint2*>(a.O + at) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

}  // namespace

}  // namespace dfl
