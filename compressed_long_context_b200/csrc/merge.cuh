// merge.cuh -- second pass of hca_decode_quant and hca_decode_shared: the partial records of each
// unit (sequence, KV head) merged by log-sum-exp, normalised, gated, mixed across heads (Virtual Head
// Attention) and stored in bf16 (or fp32).
//
// A record is what one CTA gathered for one unit: per head a reference m (log2 units), the sum l of
// 2^(z - m) and the 512 sums of 2^(z - m) v.  hca_decode_shared adds a second kind: the shared prefix
// of 2 * (128 / G) sequences at once.
//
// Grid (units, 512 / CH): a CTA owns all G heads of one unit for CH channels, so the mixing across heads stays on chip.
// Thread = (4 channels, kHeads heads): a warp reads whole 128-byte lines of four heads (CH = 32) or 32-byte sectors of 16
// (CH = 8).  The records of a chunk are all loaded before any is used (one memory round trip for up to kChunk of
// them).  What bounds it: the records, which lie in L2, and two dependent round trips.
#pragma once

#include "decode.cuh"

namespace hca {

// hca_decode_shared's two passes share the GPU: how many clusters of four SMs attend the prefix, and how many CTAs
// the sequences' own tiles.  Both passes, and the host for their grids, compute it from the same numbers.
struct SharedPlan {
    int clusters, splits;
};

// pfx: prefix tiles (256 rows x 256 keys); own: own tiles (128 keys of one sequence) of `units` (sequence, KV head)
// pairs.  The plan with the shortest longer pass, from measured times (tenths of a microsecond): a prefix tile takes a
// cluster 3.1 us after 14 us of start and record; the own pass takes 10 us and 2.5 us for each tile, of which a unit's start
// counts as two (decode_quant.cuh), in a CTA, and 6 us more where CTAs hold parts of several units.
__host__ __device__ inline long long shared_time(long long pfx, long long own, int units, int c, int sms) {
    const int ns = sms - 4 * c;
    if (c > pfx || ns < 4) return 0x3fffffffffffffLL;
    const long long tp = 140 + 31 * ((pfx + c - 1) / c);
    const long long ts = 100 + 25 * ((own + 2LL * units + ns - 1) / ns) + (units > ns ? 60 : 0);
    return tp > ts ? tp : ts;
}
inline SharedPlan shared_plan(long long pfx, long long own, int units, int max_clusters, int sms) {
    int best = 1;
    for (int c = 2; c <= max_clusters; ++c)
        if (shared_time(pfx, own, units, c, sms) < shared_time(pfx, own, units, best, sms)) best = c;
    return SharedPlan{best, sms - 4 * best};
}
// The same by a whole warp (up to 255 clusters), on every lane.
__device__ __forceinline__ SharedPlan shared_plan_warp(long long pfx, long long own, int units, int max_clusters, int sms) {
    long long key = 0x7fffffffffffffffLL;          // (time, clusters)
    for (int c = (threadIdx.x & 31) + 1; c <= max_clusters; c += 32) {
        const long long k = shared_time(pfx, own, units, c, sms) << 8 | c;
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

constexpr float kLowest = -3.402823466e38f;     // the lowest finite reference

template <int CH>
struct MergeShape {
    static constexpr int kThreads = CH == 32 ? 256 : 128;
    static constexpr int kStep = kThreads / (CH / 4);         // a thread's heads are this far apart
    static constexpr int kHeads = kDecHeads / kStep;          // heads per thread
};
template <int CH>
constexpr uint32_t merge_vha_smem(int r) {
    return (uint32_t)(2 * kDecHeads * r + kDecHeads * CH + r * CH) * 4u;
}

template <int kChunk, int CH, bool kVha, bool kPfx>
__global__ void __launch_bounds__(MergeShape<CH>::kThreads) merge_kernel(const MergeParams p) {
    constexpr int kMergeThreads = MergeShape<CH>::kThreads, kMergeStep = MergeShape<CH>::kStep, kMergeHeads = MergeShape<CH>::kHeads;
    constexpr int kLanes = CH / 4;                    // threads of one head
    extern __shared__ float cs[];
    const int u = blockIdx.x;
    const int hb = threadIdx.x / kLanes;
    const int c4 = 4 * (threadIdx.x % kLanes);
    const int c = blockIdx.y * CH + c4;                       // channels c .. c+3
    const int b = p.Hkv == 1 ? u : u / p.Hkv, g = u - b * p.Hkv;
    const size_t orow = ((size_t)b * p.Hq + (size_t)g * p.G + hb) * kDecD + c;
    const int R = p.vha_r;
    float* os = cs;                                   // [64][CH] merged, gated outputs (16-byte rows)
    float* ts = os + kDecHeads * CH;                  // [R][CH]  V^T o
    float* vs = ts + R * CH;                          // [G][R]
    float* us = vs + kDecHeads * R;                   // [G][R]
    // the inputs are not products of the passes before: read ahead of the wait for their last writes (this grid starts when
    // their CTAs have left)
    uint2 graw[kMergeHeads];
#pragma unroll
    for (int x = 0; x < kMergeHeads; ++x) {
        graw[x] = make_uint2(0, 0);
        if (p.gate && hb + kMergeStep * x < p.G) graw[x] = __ldg(reinterpret_cast<const uint2*>(p.gate + orow + (size_t)kMergeStep * x * kDecD));
    }
    const int len = __ldg(p.seqlens + b);
    if (kVha) {
        for (int i = threadIdx.x; i < p.G * R; i += kMergeThreads) {
            vs[i] = __ldg(p.vha_v + i);
            us[i] = __ldg(p.vha_u + i);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float4 r[kMergeHeads];
    // requested together: a second round trip then brings the records
    const unsigned err = __ldcg(&g_error);
    const int first = __ldcg(p.meta + 2 * u), last = __ldcg(p.meta + 2 * u + 1);
    const int clusters = kPfx ? __ldcg(&p.plan->clusters) : 0;
    if (gave_up(err)) {
        // a CTA gave up: its records may be stale, so the outputs are marked invalid
#pragma unroll
        for (int x = 0; x < kMergeHeads; ++x) r[x] = make_float4(NAN, NAN, NAN, NAN);
    } else if (len <= 0) {
        // a padding row (length 0; negative lengths are reported by the first pass)
#pragma unroll
        for (int x = 0; x < kMergeHeads; ++x) r[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
        float M[kMergeHeads], L[kMergeHeads];
#pragma unroll
        for (int x = 0; x < kMergeHeads; ++x) {
            M[x] = -INFINITY;
            L[x] = 0.f;
            r[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // records rec0 + first .. rec0 + last of `stride` rows, of which this unit's heads start at `row`
        auto fold = [&](const float* pm, const float* pl, const float* po, int first, int last, size_t rec0, int row, int stride) {
#pragma unroll 1
            for (int i0 = first; i0 <= last; i0 += kChunk) {
                float m[kChunk][kMergeHeads], l[kChunk][kMergeHeads];
                float4 o[kChunk][kMergeHeads];
#pragma unroll
                for (int k = 0; k < kChunk; ++k)
#pragma unroll
                    for (int x = 0; x < kMergeHeads; ++x) {
                        // ranges are contiguous: every record is there
                        const bool ok = hb + kMergeStep * x < p.G && i0 + k <= last;
                        const size_t rec = (rec0 + (size_t)(i0 + k)) * stride + row + hb + kMergeStep * x;
                        m[k][x] = ok ? __ldcg(pm + rec) : -INFINITY;
                        l[k][x] = ok ? __ldcg(pl + rec) : 0.f;
                        o[k][x] = ok ? __ldcg(reinterpret_cast<const float4*>(po + rec * kDecD + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                for (int x = 0; x < kMergeHeads; ++x) {
                    float Mn = M[x];
#pragma unroll
                    for (int k = 0; k < kChunk; ++k) Mn = fmaxf(Mn, m[k][x]);
                    if (Mn == -INFINITY) continue;
                    const float sc = M[x] == -INFINITY ? 0.f : exp2f(M[x] - Mn);
                    L[x] *= sc;
                    r[x] = make_float4(r[x].x * sc, r[x].y * sc, r[x].z * sc, r[x].w * sc);
#pragma unroll
                    for (int k = 0; k < kChunk; ++k) {
                        // a record without a visible key (m = -inf) holds nothing: its sums are not used (one whose
                        // keys all have logits of -inf or NaN has m = kLowest: it weighs nothing, or makes the row NaN)
                        if (m[k][x] == -INFINITY) continue;
                        const float w = exp2f(m[k][x] - Mn);
                        L[x] = fmaf(w, l[k][x], L[x]);
                        r[x].x = fmaf(w, o[k][x].x, r[x].x);
                        r[x].y = fmaf(w, o[k][x].y, r[x].y);
                        r[x].z = fmaf(w, o[k][x].z, r[x].z);
                        r[x].w = fmaf(w, o[k][x].w, r[x].w);
                    }
                    M[x] = Mn;
                }
            }
        };
        if (first < 0 || last < first || last >= p.nsplit) {
            if (threadIdx.x == 0 && blockIdx.y == 0) record_error(HCA_ERR_DEVICE_INPUT);
        } else {
            fold(p.rec_m, p.rec_l, p.rec_o, first, last, (size_t)u, 0, kDecHeads);
        }
        if (kPfx && p.pfx_tiles > 0) {
            const int rt = (b / (2 * p.tpt)) * p.Hkv + g;
            const long long per = pfx_per(p.pfx_total, min(clusters, p.pfx_clusters));
            const int pf = (int)((long long)rt * p.pfx_tiles / per);
            const int pl = (int)(((long long)(rt + 1) * p.pfx_tiles - 1) / per);
            fold(p.pfx_m, p.pfx_l, p.pfx_o, pf, pl, (size_t)rt, (b / p.tpt & 1) * 128 + (b % p.tpt) * p.G, 256);
        }
#pragma unroll
        for (int x = 0; x < kMergeHeads; ++x) {
            const float inv = 1.f / L[x];
            r[x] = make_float4(r[x].x * inv, r[x].y * inv, r[x].z * inv, r[x].w * inv);
            if (p.gate) {
                r[x].x *= __frcp_rn(1.f + __expf(-bf16lo(graw[x].x)));
                r[x].y *= __frcp_rn(1.f + __expf(-bf16hi(graw[x].x)));
                r[x].z *= __frcp_rn(1.f + __expf(-bf16lo(graw[x].y)));
                r[x].w *= __frcp_rn(1.f + __expf(-bf16hi(graw[x].y)));
            }
        }
    }
    if (kVha) {
        // o'[:, ch] = o[:, ch] + U (V^T o[:, ch]) over the G heads of this token (see decode.cuh)
#pragma unroll
        for (int x = 0; x < kMergeHeads; ++x)
            if (hb + kMergeStep * x < p.G) *reinterpret_cast<float4*>(os + (hb + kMergeStep * x) * CH + c4) = r[x];
        __syncthreads();
        for (int i = threadIdx.x; i < R * kLanes; i += kMergeThreads) {
            const int k = i / kLanes, cc = (i % kLanes) * 4;
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int hd = 0; hd < p.G; ++hd) {
                const float vk = vs[hd * R + k];
                const float4 o4 = *reinterpret_cast<const float4*>(os + hd * CH + cc);
                t.x = fmaf(vk, o4.x, t.x);
                t.y = fmaf(vk, o4.y, t.y);
                t.z = fmaf(vk, o4.z, t.z);
                t.w = fmaf(vk, o4.w, t.w);
            }
            *reinterpret_cast<float4*>(ts + k * CH + cc) = t;
        }
        __syncthreads();
        for (int k = 0; k < R; ++k) {
            const float4 t4 = *reinterpret_cast<const float4*>(ts + k * CH + c4);
#pragma unroll
            for (int x = 0; x < kMergeHeads; ++x) {
                if (hb + kMergeStep * x >= p.G) continue;
                const float uk = us[(hb + kMergeStep * x) * R + k];
                r[x].x = fmaf(uk, t4.x, r[x].x);
                r[x].y = fmaf(uk, t4.y, r[x].y);
                r[x].z = fmaf(uk, t4.z, r[x].z);
                r[x].w = fmaf(uk, t4.w, r[x].w);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < kMergeHeads; ++x) {
        if (hb + kMergeStep * x >= p.G) continue;
        const size_t at = orow + (size_t)kMergeStep * x * kDecD;
        if (p.out_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = r[x];
        else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
                make_uint2(pack_bf16x2(r[x].x, r[x].y), pack_bf16x2(r[x].z, r[x].w));
    }
}

}  // namespace hca
