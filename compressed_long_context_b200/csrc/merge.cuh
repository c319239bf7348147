// merge.cuh -- second pass of hca_decode_quant and hca_decode_shared: the partial records of each
// unit (sequence, KV head) merged by log-sum-exp, normalised, gated, mixed across heads (Virtual Head
// Attention) and stored in bf16 (or fp32).
//
// A record is what one CTA gathered for one unit: per head a reference m (log2 units), the sum l of
// 2^(z - m) and the 512 sums of 2^(z - m) v.  hca_decode_shared adds a second kind: the shared prefix
// of 2 * (128 / G) sequences at once.
//
// Grid (units, 512 / 32), 128 threads: a CTA owns all G heads of one unit for 32 channels, thread =
// (head, 16 channels), so the mixing across heads stays on chip.  The records of a chunk are all
// loaded before any is used (one memory round trip for up to kChunk of them).
#pragma once

#include "decode.cuh"

namespace hca {

// hca_decode_shared's two passes share the GPU: how many clusters of four SMs attend the prefix, and how many CTAs
// the sequences' own tiles.  Both passes, and the host for their grids, compute it from the same numbers.
struct SharedPlan {
    int clusters, splits;
};

// pfx: prefix tiles (256 rows x 256 keys); own: own tiles (128 keys of one sequence).  The plan with the shortest longer
// pass, from measured times: a prefix tile takes a cluster about 2.8 us after 14 us of start and record, an own tile
// takes one SM (its loads' latency) about 4 us after 18 us.
__host__ __device__ inline long long shared_time(long long pfx, long long own, int c, int sms) {
    const int ns = sms - 4 * c;
    if (c > pfx || ns < 4) return 0x3fffffffffffffLL;
    const long long tp = 140 + 28 * ((pfx + c - 1) / c), ts = 180 + 40 * ((own + ns - 1) / ns);
    return tp > ts ? tp : ts;
}
inline SharedPlan shared_plan(long long pfx, long long own, int max_clusters, int sms) {
    int best = 1;
    for (int c = 2; c <= max_clusters; ++c)
        if (shared_time(pfx, own, c, sms) < shared_time(pfx, own, best, sms)) best = c;
    return SharedPlan{best, sms - 4 * best};
}
// The same by a whole warp (up to 255 clusters), on every lane.
__device__ __forceinline__ SharedPlan shared_plan_warp(long long pfx, long long own, int max_clusters, int sms) {
    long long key = 0x7fffffffffffffffLL;          // (time, clusters)
    for (int c = (threadIdx.x & 31) + 1; c <= max_clusters; c += 32) {
        const long long k = shared_time(pfx, own, c, sms) << 8 | c;
        key = k < key ? k : key;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const long long k = __shfl_xor_sync(0xffffffffu, key, off);
        key = k < key ? k : key;
    }
    const int c = (int)(key & 255);
    return SharedPlan{c, sms - 4 * c};
}

// Prefix tiles in one cluster's range.
__host__ __device__ inline long long pfx_per(long long total, int clusters) { return (total + clusters - 1) / clusters; }

struct MergeParams {
    const int* seqlens;           // [B]
    const int* meta;              // [U][2]: first and last CTA holding a piece of unit u
    const float* rec_m;           // [R][64]
    const float* rec_l;           // [R][64]
    const float* rec_o;           // [R][64][512]
    const float* pfx_m;           // [RP][256] prefix records (hca_decode_shared), or null
    const float* pfx_l;           // [RP][256]
    const float* pfx_o;           // [RP][256][512]
    const __nv_bfloat16* gate;    // [B, Hq, 512] or null
    const float* vha_u;           // [Hq, vha_r] or null
    const float* vha_v;
    void* out;                    // [B, Hq, 512]
    int vha_r, B, Hq, Hkv, G, nsplit, out_f32;
    // prefix records: a row tile holds 2 tpt sequences of one KV head, 128 rows for each tpt of them; its key tiles are
    // numbers [rt * pfx_tiles, (rt + 1) * pfx_tiles) of the list that is cut into one range per cluster of the plan
    int tpt, pfx_tiles, pfx_clusters;
    long long pfx_total;
    const SharedPlan* plan;
};

template <int kChunk, bool kVha, bool kPfx>
__global__ void __launch_bounds__(128) merge_kernel(const MergeParams p) {
    extern __shared__ float cs[];
    const int u = blockIdx.x;
    const int h = threadIdx.x >> 1;
    const int c16 = 16 * (threadIdx.x & 1);
    const int c = blockIdx.y * kMergeCh + c16;                      // channels c .. c+15
    const int b = u / p.Hkv, g = u - (u / p.Hkv) * p.Hkv;
    const bool live = h < p.G;
    const size_t orow = ((size_t)b * p.Hq + (size_t)g * p.G + (live ? h : 0)) * kDecD + c;
    const int R = p.vha_r;
    float* os = cs;                                   // [64][32] merged, gated outputs (16-byte rows)
    float* ts = os + kDecHeads * kMergeCh;            // [R][32]  V^T o
    float* vs = ts + R * kMergeCh;                    // [G][R]
    float* us = vs + kDecHeads * R;                   // [G][R]
    // the inputs are not products of the passes before: read while those still run
    uint4 graw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (p.gate && live) {
        graw[0] = __ldg(reinterpret_cast<const uint4*>(p.gate + orow));
        graw[1] = __ldg(reinterpret_cast<const uint4*>(p.gate + orow) + 1);
    }
    const int len = __ldg(p.seqlens + b);
    if (kVha) {
        for (int i = threadIdx.x; i < p.G * R; i += 128) {
            vs[i] = __ldg(p.vha_v + i);
            us[i] = __ldg(p.vha_u + i);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float r[16];
    if (*reinterpret_cast<volatile unsigned int*>(&g_error) == HCA_ERR_TIMEOUT) {
        // a CTA gave up: its records may be stale, so the outputs are marked invalid
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = NAN;
    } else if (len <= 0) {
        // a padding row (length 0; negative lengths are reported by the first pass)
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = 0.f;
    } else {
        float M = -INFINITY, L = 0.f;
        float acc[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[j] = 0.f;
        // `kind` 0: the unit's own records; 1: the prefix records of its row tile
        auto fold = [&](int kind, int first, int last, size_t rec0, int row, int stride) {
            const float* pm = kind ? p.pfx_m : p.rec_m;
            const float* pl = kind ? p.pfx_l : p.rec_l;
            const float* po = kind ? p.pfx_o : p.rec_o;
            for (int i0 = first; i0 <= last; i0 += kChunk) {
                float m[kChunk], l[kChunk];
                float4 o[kChunk][4];
#pragma unroll
                for (int k = 0; k < kChunk; ++k) {
                    const bool ok = live && i0 + k <= last;   // ranges are contiguous: every one has a record
                    const size_t rec = (rec0 + (size_t)(i0 + k)) * stride + row;
                    m[k] = ok ? __ldcg(pm + rec) : -INFINITY;
                    l[k] = ok ? __ldcg(pl + rec) : 0.f;
                    const float4* op = reinterpret_cast<const float4*>(po + rec * kDecD + c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[k][j] = ok ? __ldcg(op + j) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                float Mn = M;
#pragma unroll
                for (int k = 0; k < kChunk; ++k) Mn = fmaxf(Mn, m[k]);
                if (Mn == -INFINITY) continue;
                const float sc = M == -INFINITY ? 0.f : exp2f(M - Mn);
                L *= sc;
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[j] *= sc;
#pragma unroll
                for (int k = 0; k < kChunk; ++k) {
                    // a record without a visible key (m = -inf) holds nothing: its sums are not used
                    if (m[k] == -INFINITY) continue;
                    const float w = exp2f(m[k] - Mn);
                    L = fmaf(w, l[k], L);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[4 * j] = fmaf(w, o[k][j].x, acc[4 * j]);
                        acc[4 * j + 1] = fmaf(w, o[k][j].y, acc[4 * j + 1]);
                        acc[4 * j + 2] = fmaf(w, o[k][j].z, acc[4 * j + 2]);
                        acc[4 * j + 3] = fmaf(w, o[k][j].w, acc[4 * j + 3]);
                    }
                }
                M = Mn;
            }
        };
        const int hh = live ? h : 0;
        const int first = __ldcg(p.meta + 2 * u), last = __ldcg(p.meta + 2 * u + 1);
        if (first < 0 || last < first || last >= p.nsplit) {
            if (threadIdx.x == 0 && blockIdx.y == 0) record_error(HCA_ERR_DEVICE_INPUT);
        } else {
            fold(0, first, last, (size_t)u, hh, kDecHeads);
        }
        if (kPfx && p.pfx_tiles > 0) {
            const int rt = (b / (2 * p.tpt)) * p.Hkv + g;
            const long long per = pfx_per(p.pfx_total, min(__ldcg(&p.plan->clusters), p.pfx_clusters));
            const int pf = (int)((long long)rt * p.pfx_tiles / per);
            const int pl = (int)(((long long)(rt + 1) * p.pfx_tiles - 1) / per);
            fold(1, pf, pl, (size_t)rt, (b / p.tpt & 1) * 128 + (b % p.tpt) * p.G + hh, 256);
        }
        const float inv = 1.f / L;
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = acc[j] * inv;
        if (p.gate) {
            const uint32_t gw[8] = {graw[0].x, graw[0].y, graw[0].z, graw[0].w,
                                    graw[1].x, graw[1].y, graw[1].z, graw[1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[2 * j] *= __frcp_rn(1.f + __expf(-bf16lo(gw[j])));
                r[2 * j + 1] *= __frcp_rn(1.f + __expf(-bf16hi(gw[j])));
            }
        }
    }
    if (kVha) {
        // o'[:, ch] = o[:, ch] + U (V^T o[:, ch]) over the G heads of this token (see decode.cuh)
        if (h < kDecHeads) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4*>(os + h * kMergeCh + c16 + 4 * j) =
                    live ? make_float4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3])
                         : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < R * (kMergeCh / 4); i += 128) {
            const int k = i >> 3, c4 = (i & 7) * 4;
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int hd = 0; hd < p.G; ++hd) {
                const float vk = vs[hd * R + k];
                const float4 o4 = *reinterpret_cast<const float4*>(os + hd * kMergeCh + c4);
                t.x = fmaf(vk, o4.x, t.x);
                t.y = fmaf(vk, o4.y, t.y);
                t.z = fmaf(vk, o4.z, t.z);
                t.w = fmaf(vk, o4.w, t.w);
            }
            *reinterpret_cast<float4*>(ts + k * kMergeCh + c4) = t;
        }
        __syncthreads();
        if (live) {
            for (int k = 0; k < R; ++k) {
                const float uk = us[h * R + k];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 t4 = *reinterpret_cast<const float4*>(ts + k * kMergeCh + c16 + 4 * j);
                    r[4 * j] = fmaf(uk, t4.x, r[4 * j]);
                    r[4 * j + 1] = fmaf(uk, t4.y, r[4 * j + 1]);
                    r[4 * j + 2] = fmaf(uk, t4.z, r[4 * j + 2]);
                    r[4 * j + 3] = fmaf(uk, t4.w, r[4 * j + 3]);
                }
            }
        }
    }
    if (!live) return;
    if (p.out_f32) {
        float* o = static_cast<float*>(p.out) + orow;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4*>(o + 4 * j) = make_float4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
    } else {
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            o[j] = make_uint4(pack_bf16x2(r[8 * j], r[8 * j + 1]), pack_bf16x2(r[8 * j + 2], r[8 * j + 3]),
                              pack_bf16x2(r[8 * j + 4], r[8 * j + 5]), pack_bf16x2(r[8 * j + 6], r[8 * j + 7]));
    }
}

}  // namespace hca
