// quant.cuh -- the 8-bit compressed cache: written from raw tokens (hca_compress_quant), one token at a
// time (hca_append_quant), and read back to bf16 (hca_read_quant).  The format is in fp8.cuh.
//
// The pooled entry stays in fp32 until it is quantised: one rounding, to e4m3.
#pragma once

#include "append.cuh"
#include "compress.cuh"
#include "fp8.cuh"

namespace hca {

// Largest magnitude over the CTA's threads (every thread calls it; scratch: one float per warp).
template <int THREADS>
__device__ __forceinline__ float block_amax(float a, float* scratch) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = a;
    __syncthreads();
    a = scratch[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) a = fmaxf(a, scratch[w]);
    return a;
}

// ------------------------------------------------------------------ compress

// A block's pooling weights (all one without w) by one warp: alpha[i] = 2^-7 exp(w[i] - max w), and their sum, at most 1, in
// alpha[128].  The pooled sums are divided by it at the end, so that the tokens wait for one step less (a 128K prompt 46.9 ->
// 45.1 us); 2^-7 keeps sums of at most 128 tokens in fp32's range.
__device__ __forceinline__ void block_alpha(const float* __restrict__ w, int64_t pos0, int blk, float* alpha) {
    const int lane = threadIdx.x & 31;
    float wv[4];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int idx = lane + 32 * i;
        wv[i] = idx < blk ? (w ? w[pos0 + idx] : 0.f) : -INFINITY;
        m = fmaxf(m, wv[i]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        wv[i] = (lane + 32 * i) < blk ? expf(wv[i] - m) * 0x1p-7f : 0.f;
        s += wv[i];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < blk) alpha[lane + 32 * i] = wv[i];
    if (lane == 0) alpha[128] = s;
}

constexpr int kPoolUnroll = 8;

// One CTA per (entry, tensor): the weighted sum over `blk` rows of D channels, then the codes of the pooled vector and its
// scale.  A stream over memory: 64 KB in flight per CTA (a lone entry takes two round trips), the first rows
// requested before the weights' softmax, whose latency they cover.  K and V of an entry are separate CTAs: few entries
// fill twice the SMs.
template <int D, int THREADS>
__device__ __forceinline__ void pool_rows_quant(const __nv_bfloat16* __restrict__ src, int64_t row_stride,
                                                const float* __restrict__ w, int64_t pos0, int blk,
                                                float* __restrict__ alpha, float* __restrict__ red,
                                                float* __restrict__ scratch, uint8_t* __restrict__ dst,
                                                uint8_t* __restrict__ scale) {
    constexpr int TPR = D / 8;                   // threads per row (16 bytes each)
    constexpr int R = THREADS / TPR;        // rows in flight per pass
    const int tid = threadIdx.x;
    const int c0 = (tid % TPR) * 8;
    const int r0 = tid / TPR;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    const __nv_bfloat16* at = src + r0 * row_stride + c0;
    const int64_t step = R * row_stride;
    for (int r = r0; r - r0 < blk; r += R * kPoolUnroll) {      // the same passes for every thread
        uint4 x[kPoolUnroll];
#pragma unroll
        for (int u = 0; u < kPoolUnroll; ++u) {
            const int rr = r + u * R;
            if (rr < blk) x[u] = __ldcs(reinterpret_cast<const uint4*>(at));
            at += step;
        }
        if (r == r0) {
            if (tid < 32) block_alpha(w, pos0, blk, alpha);
            __syncthreads();
        }
        // a pass's own sums: shorter chains of roundings (codes that differ from 64-bit pooling's, of 21 million: 99 instead of
        // 130; torch's fp32 sums 121), for 0.5 of 45 us
        float part[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) part[i] = 0.f;
#pragma unroll
        for (int u = 0; u < kPoolUnroll; ++u) {
            const int rr = r + u * R;
            // a token without weight (w = -inf: padding) may hold anything
            const float a = rr < blk ? alpha[rr] : 0.f;
            if (a != 0.f) {
                part[0] = fmaf(a, bf16lo(x[u].x), part[0]);
                part[1] = fmaf(a, bf16hi(x[u].x), part[1]);
                part[2] = fmaf(a, bf16lo(x[u].y), part[2]);
                part[3] = fmaf(a, bf16hi(x[u].y), part[3]);
                part[4] = fmaf(a, bf16lo(x[u].z), part[4]);
                part[5] = fmaf(a, bf16hi(x[u].z), part[5]);
                part[6] = fmaf(a, bf16lo(x[u].w), part[6]);
                part[7] = fmaf(a, bf16hi(x[u].w), part[7]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += part[i];
    }
    // rows of one warp first (narrow rows: several to a warp), then across warps
    constexpr int RW = TPR < 32 ? 32 / TPR : 1;
#pragma unroll
    for (int off = TPR; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
    if (r0 % RW == 0) {
        float4* o = reinterpret_cast<float4*>(red + (r0 / RW) * D + c0);
        o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
    __syncthreads();
    // two channels per thread
    float s0 = 0.f, s1 = 0.f;
    const bool mine = tid < D / 2;
    if (mine) {
#pragma unroll 8
        for (int r = 0; r < R / RW; ++r) {
            const float2 p = *reinterpret_cast<const float2*>(red + r * D + 2 * tid);
            s0 += p.x;
            s1 += p.y;
        }
        s0 /= alpha[128];
        s1 /= alpha[128];
    }
    const uint32_t byte = q_scale_byte(block_amax<THREADS>(fmaxf(q_mag(s0), q_mag(s1)), scratch));
    const float inv = q_inv_scale(byte);
    if (mine) reinterpret_cast<uint16_t*>(dst)[tid] = (uint16_t)q_codes2(s0, s1, inv);
    if (tid == 0) *scale = (uint8_t)byte;
}

template <int DK, int DV, int THREADS>
__global__ void __launch_bounds__(THREADS, 768 / THREADS)
compress_quant_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                      const float* __restrict__ w, uint8_t* __restrict__ kc, uint8_t* __restrict__ vc,
                      uint8_t* __restrict__ sc, int T, int Hkv, int blk, int Nc) {
    __shared__ float alpha[129];
    __shared__ __align__(16) float red[THREADS * 8];
    __shared__ float scratch[THREADS / 32];
    const int e = blockIdx.x;                 // entry index, KV head fastest
    const int bj = e / Hkv, g = e - bj * Hkv;
    const int b = bj / Nc, j = bj - b * Nc;
    const int64_t pos0 = (int64_t)b * T + (int64_t)blk * j;
    if (blockIdx.y == 0)
        pool_rows_quant<DK, THREADS>(k + (pos0 * Hkv + g) * DK, (int64_t)Hkv * DK, w, pos0, blk, alpha, red, scratch,
                            kc + (int64_t)e * DK, sc + 2 * (int64_t)e);
    else
        pool_rows_quant<DV, THREADS>(v + (pos0 * Hkv + g) * DV, (int64_t)Hkv * DV, w, pos0, blk, alpha, red, scratch,
                            vc + (int64_t)e * DV, sc + 2 * (int64_t)e + 1);
}

// ------------------------------------------------------------------ append

struct AppendQuantParams {
    const __nv_bfloat16* k_new;   // [B, Hkv, d]
    const __nv_bfloat16* v_new;   // [B, Hkv, dv]
    const float* w;               // [B] or null (weight 0)
    const int* seqlens;           // [B], length including the new token; 0: a padding row
    __nv_bfloat16* kw;            // [B, W, Hkv, d] ring
    __nv_bfloat16* vw;
    uint8_t* kc;                  // [B, Nmax, Hkv, d] codes or pool [P, ps, Hkv, d]
    uint8_t* vc;
    uint16_t* sc;                 // [B, Nmax, Hkv] or [P, ps, Hkv] scale pairs
    const int* page_table;        // [B, max_pages] or null
    float* state;                 // [B, Hkv, kAppendHeader + d + dv]
    int B, Hkv, d, dv, blk, W, Nmax, page_size, max_pages, num_pages;
};

// One CTA per (sequence, KV head), thread i owns channels 4i .. 4i+3 of K and of V, as append_kernel;
// every load is issued before any result is needed, so a call costs one memory round trip.  Completing a
// block adds two block-wide maxima.
__global__ void __launch_bounds__(kAppendThreads) append_quant_kernel(const AppendQuantParams p) {
    __shared__ float scratch[2][kAppendThreads / 32];
    const int u = blockIdx.x;
    const int b = u / p.Hkv, g = u - b * p.Hkv;
    const int c = 4 * threadIdx.x;
    const bool hk = c < p.d, hv = c < p.dv;
    float* st = p.state + (size_t)u * (kAppendHeader + p.d + p.dv);
    float* acc_k = st + kAppendHeader;
    float* acc_v = st + kAppendHeader + p.d;
    const int L = __ldg(p.seqlens + b);
    const float w = p.w ? __ldg(p.w + b) : 0.f;
    const float2 ms = *reinterpret_cast<const float2*>(st);
    const uint2 xk = hk ? *reinterpret_cast<const uint2*>(p.k_new + (size_t)u * p.d + c) : make_uint2(0u, 0u);
    const uint2 xv = hv ? *reinterpret_cast<const uint2*>(p.v_new + (size_t)u * p.dv + c) : make_uint2(0u, 0u);
    float4 tk = hk ? *reinterpret_cast<const float4*>(acc_k + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 tv = hv ? *reinterpret_cast<const float4*>(acc_v + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (L < 1) {
        if (L < 0 && threadIdx.x == 0) record_error(HCA_ERR_DEVICE_INPUT);
        return;
    }
    const long long pos = (long long)L - 1;
    const int slot = (int)(pos % p.W);
    const float m_old = ms.x, s_old = ms.y;
    // a weight of -inf adds nothing, also as a block's first; NaN stays in the sum until the block is complete
    const bool empty = s_old == 0.f;
    const float m_new = empty ? w : fmaxf(m_old, w);
    const float a = empty ? 0.f : expf(m_old - m_new);
    const float e = w == -INFINITY ? 0.f : expf(w - m_new);
    const float s_new = fmaf(s_old, a, e);
    const bool complete = (pos + 1) % p.blk == 0;
    auto fold = [&](uint2 x, float4& t) {
        if (e == 0.f) x = make_uint2(0u, 0u);       // a token without weight may hold anything
        t.x = fmaf(e, bf16lo(x.x), t.x * a);
        t.y = fmaf(e, bf16hi(x.x), t.y * a);
        t.z = fmaf(e, bf16lo(x.y), t.z * a);
        t.w = fmaf(e, bf16hi(x.y), t.w * a);
    };
    const size_t ring = ((size_t)b * p.W + slot) * p.Hkv + g;
    fold(xk, tk);
    fold(xv, tv);
    if (hk) *reinterpret_cast<uint2*>(p.kw + ring * p.d + c) = xk;
    if (hv) *reinterpret_cast<uint2*>(p.vw + ring * p.dv + c) = xv;
    if (complete) {
        const float inv_s = 1.f / s_new;
        const float4 ek = make_float4(tk.x * inv_s, tk.y * inv_s, tk.z * inv_s, tk.w * inv_s);
        const float4 ev = make_float4(tv.x * inv_s, tv.y * inv_s, tv.z * inv_s, tv.w * inv_s);
        auto amax4 = [](float4 x) { return fmaxf(fmaxf(q_mag(x.x), q_mag(x.y)), fmaxf(q_mag(x.z), q_mag(x.w))); };
        const uint32_t kb = q_scale_byte(block_amax<kAppendThreads>(hk ? amax4(ek) : 0.f, scratch[0]));
        const uint32_t vb = q_scale_byte(block_amax<kAppendThreads>(hv ? amax4(ev) : 0.f, scratch[1]));
        // the entry's row (none: out of the cache, reported)
        const long long j = pos / p.blk;
        long long row = -1;
        if (p.page_table) {
            const long long pi = j / p.page_size;
            if (pi < p.max_pages) {
                const int pg = __ldg(p.page_table + (size_t)b * p.max_pages + pi);
                if (pg >= 0 && pg < p.num_pages) row = (long long)pg * p.page_size + j % p.page_size;
            }
        } else if (j < p.Nmax) {
            row = (long long)b * p.Nmax + j;
        }
        if (row >= 0) {
            const size_t rg = (size_t)row * p.Hkv + g;
            if (hk) *reinterpret_cast<uint32_t*>(p.kc + rg * p.d + c) = q_codes4(ek, q_inv_scale(kb));
            if (hv) *reinterpret_cast<uint32_t*>(p.vc + rg * p.dv + c) = q_codes4(ev, q_inv_scale(vb));
            if (threadIdx.x == 0) p.sc[rg] = (uint16_t)(kb | vb << 8);
        } else if (threadIdx.x == 0) {
            record_error(HCA_ERR_DEVICE_INPUT);
        }
        tk = tv = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (hk) *reinterpret_cast<float4*>(acc_k + c) = tk;
    if (hv) *reinterpret_cast<float4*>(acc_v + c) = tv;
    __syncthreads();      // every thread has read m and s
    if (threadIdx.x == 0) *reinterpret_cast<float2*>(st) = complete ? make_float2(0.f, 0.f) : make_float2(m_new, s_new);
}

// ------------------------------------------------------------------ read back

struct ReadQuantParams {
    const uint8_t* kc;            // [B, Nmax, Hkv, d] codes or pool [P, ps, Hkv, d]
    const uint8_t* vc;
    const uint16_t* sc;
    const int* page_table;        // [B, max_pages] or null
    const int* counts;            // [B] entries to read
    __nv_bfloat16* k;             // [B, n, Hkv, d]
    __nv_bfloat16* v;
    int B, n, Hkv, d, dv, Nmax, page_size, max_pages, num_pages;
    long long items;              // B * n * Hkv
};

constexpr int kReadThreads = 256;

// One warp per (sequence, entry, KV head): 16 codes per lane and step, two 16-byte stores.  Entries at and
// past counts[b] are left as they are.
__global__ void __launch_bounds__(kReadThreads) read_quant_kernel(const ReadQuantParams p) {
    const int lane = threadIdx.x & 31;
    const long long nw = (long long)gridDim.x * (kReadThreads / 32);
    for (long long i = (long long)blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5); i < p.items; i += nw) {
        const int g = (int)(i % p.Hkv);
        const long long bj = i / p.Hkv;
        const int j = (int)(bj % p.n);
        const int b = (int)(bj / p.n);
        const long long cap = p.page_table ? (long long)p.max_pages * p.page_size : (long long)p.Nmax;
        const int cnt = __ldg(p.counts + b);
        if ((cnt < 0 || cnt > p.n || cnt > cap) && j == 0 && lane == 0) record_error(HCA_ERR_DEVICE_INPUT);
        if (j >= cnt || j >= cap) continue;
        long long row = (long long)b * p.Nmax + j;
        if (p.page_table) {
            const int pg = __ldg(p.page_table + (size_t)b * p.max_pages + j / p.page_size);
            if (pg < 0 || pg >= p.num_pages) {
                if (lane == 0) record_error(HCA_ERR_DEVICE_INPUT);
                continue;
            }
            row = (long long)pg * p.page_size + j % p.page_size;
        }
        const size_t rg = (size_t)row * p.Hkv + g;
        const uint32_t sc = __ldg(p.sc + rg);
        auto widen = [&](const uint8_t* src, __nv_bfloat16* dst, int D, float s) {
            for (int c = 16 * lane; c < D; c += 512) {
                const uint4 x = __ldcs(reinterpret_cast<const uint4*>(src + c));
                const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
                uint32_t y[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 a = e4m3x2_f32(w4[q] & 0xffffu), b2 = e4m3x2_f32(w4[q] >> 16);
                    y[2 * q] = pack_bf16x2(a.x * s, a.y * s);
                    y[2 * q + 1] = pack_bf16x2(b2.x * s, b2.y * s);
                }
                uint4* o = reinterpret_cast<uint4*>(dst + c);
                __stcs(o, make_uint4(y[0], y[1], y[2], y[3]));
                __stcs(o + 1, make_uint4(y[4], y[5], y[6], y[7]));
            }
        };
        widen(p.kc + rg * p.d, p.k + (size_t)i * p.d, p.d, q_scale(sc & 0xffu));
        widen(p.vc + rg * p.dv, p.v + (size_t)i * p.dv, p.dv, q_scale(sc >> 8));
    }
}

}  // namespace hca
