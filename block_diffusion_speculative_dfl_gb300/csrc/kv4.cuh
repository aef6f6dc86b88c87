// Layout of the 4-bit context cache and the conversions its kernels share.
//
// A cached element is c * s * 2^e: c an e2m1 code, s an e4m3 scale of 16
// consecutive dimensions of one token, e an integer of the pool.  c * s has at
// most 6 significant bits and lies in {0} or [2^-10, 2688], so it is exact in
// fp16 and in bf16: reading a cell rounds nothing.
//
// Cell: 16 consecutive tokens of one K/V head, the unit of a page (a page of P
// tokens is [Hkv][P/16] cells) and of the attention's copies.  Its bytes are
//   K codes  [16 rows][hd/2]   row = slot of the token, two dims per byte
//   K scales [16 * hd/16]      in the order of the lanes that use them
//   V codes  [16 rows][hd/2]   row = token
//   V scales [hd/16][16]       four tokens of one lane side by side
// The orders serve the attention kernel's fragments (kv4_attn.cu): lane
// (g, t) = (lane / 4, lane % 4) of a warp reads the K codes of slots g and
// g + 8 at quarter t of the head, their scales as one word, and the V codes
// of tokens t, 4 + t, 8 + t, 12 + t (slots 2t, 2t + 1, 2t + 8, 2t + 9 of the
// products) at eighth g, their scales as one word; every such access of a
// warp is free of bank conflicts.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dfl {

constexpr int KV4_CELL_TOKENS = 16;

template <int HD>
struct Kv4Cell {
    static_assert(HD == 64 || HD == 128, "head dim");
    static constexpr int ROW = HD / 2;                   // bytes of a token's codes
    static constexpr int GROUPS = HD / 16;
    static constexpr int K_CODES = 0;
    static constexpr int K_SCALES = 16 * ROW;
    static constexpr int V_CODES = K_SCALES + 16 * GROUPS;
    static constexpr int V_SCALES = V_CODES + 16 * ROW;
    static constexpr int BYTES = V_SCALES + 16 * GROUPS;   // 18 * HD, a multiple of 16

    // token 8h + 4i + t sits at slot 8h + 2t + i
    static __device__ __forceinline__ int slot(int tok) { return (tok & 8) + 2 * (tok & 3) + ((tok >> 2) & 1); }
    static __device__ __forceinline__ int token(int slot) { return (slot & 8) + 4 * (slot & 1) + ((slot & 7) >> 1); }
    static __device__ __forceinline__ int k_code(int tok, int group) { return K_CODES + slot(tok) * ROW + group * 8; }
    static __device__ __forceinline__ int k_scale(int tok, int group) {
        constexpr int GPT = HD / 64;   // groups of a lane's quarter
        const int s = slot(tok);
        return K_SCALES + (((s & 7) * 4 + group / GPT) * 2 + (s >> 3)) * GPT + group % GPT;
    }
    // hd = 128: the halves of a row trade places in every other pair of tokens,
    // so that four tokens' reads of the same eighth fall into different banks
    static __device__ __forceinline__ int v_swap(int tok) { return HD == 128 && (tok & 2) ? ROW / 2 : 0; }
    static __device__ __forceinline__ int v_code(int tok, int group) {
        return V_CODES + tok * ROW + ((group * 8) ^ v_swap(tok));
    }
    static __device__ __forceinline__ int v_scale(int tok, int group) {
        return V_SCALES + group * 16 + (tok & 3) * 4 + (tok >> 2);
    }
};

// The pool as the kernels see it: one layer's slab.
struct Kv4Slab {
    uint8_t* data;          // [num_pages][Hkv][page / 16] cells
    int num_pages, page, Hkv;
    int cells;              // cells of a page and head
};

// 2^e as a float, -126 <= e <= 127.
__host__ __device__ __forceinline__ float kv4_exp2i(int e) {
#ifdef __CUDA_ARCH__
    return __int_as_float((e + 127) << 23);
#else
    return e >= 0 ? (float)(1ull << (e < 63 ? e : 63)) : 1.0f / (float)(1ull << (-e < 63 ? -e : 63));
#endif
}

// Four bytes of e2m1 pairs -> four fp16 pairs (low nibble in the low half).
__device__ __forceinline__ void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// Two e4m3 bytes (low 16 bits) -> an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_half(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 b;\n\tcvt.u16.u32 b, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(h) : "r"(w));
    return h;
}

__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Pairwise maximum of two 16-bit unsigned numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Block-wide sums over per-sequence unit counts, shared by the kernels that
// cut a ragged batch into equal ranges.
// Exclusive prefix of v over the block's threads; total in *sum.  `red` holds
// one value per warp.  All threads call; ends with the block synchronised.
template <int THREADS, typename T>
__device__ __forceinline__ T block_exscan(T v, T* red, T* sum) {
    constexpr int W = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = v;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    T all = lane < W ? red[lane] : 0;   // every warp sums the warps' totals
    const T own = all;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xFFFFFFFFu, all, o);
        if (lane >= o) all += u;
    }
    const T before = __shfl_sync(0xFFFFFFFFu, all - own, warp);
    *sum = __shfl_sync(0xFFFFFFFFu, all, W - 1);
    __syncthreads();
    return before + inc - v;
}

}  // namespace dfl
