// prefix.cuh -- attention of a batch's queries to the entries that all its sequences share
// (first pass of hca_decode_shared).
//
// A common prefix of Np entries is held once.  The 64 heads of one sequence fill half an MMA tile and read every
// entry; here the heads of four sequences (2 tpt with tpt = 128 / G) stand in one tile of 256 rows, and every
// entry is read from L2 once per row tile instead of from memory once per sequence:
//   z[r, j] = scale q_r . k_j   over the entries j < min(Np, n_c) that row r's sequence sees,
// one softmax per row over a range of key tiles, kept as a record (reference m, l = sum 2^(z - m), O = sum 2^(z - m) v)
// that merge.cuh joins with those of the row's own entries and window.
//
// The list of (row tile, key tile of 256 entries) pairs, row tile by row tile, is cut into one range per
// cluster of four SMs, which share the work by stage, as prefill_pair.cuh does, and by rows:
//   ranks 0, 1 (S pair)  S = Q K^T and softmax: M = 256, N = 256 MMAs of the pair (cta_group::2), each SM with its
//                        128 rows of Q and of S, and half of every K slab;
//   ranks 2, 3 (O pair)  O += P V, M = 256, N = 256 value columns, all 512 in tensor memory, each SM with its 128
//                        rows of P and of O, and half of every V slab; S rank h sends its P to O rank h.
// Why pairs: one SM's 128 x 256 x 512 products take 4096 cycles and read 256 KB of K or V, 64 bytes a cycle, more
// than L2 delivers to all SMs at once; the pair halves that.  The first MMA issuer of a pair (the leader) waits
// for both SMs' copies (they count their bytes on the leader's barrier), and its commits arrive at both.
//
// Every barrier but kPxXch is arrived at from another SM of the cluster as well, so its waits acquire at cluster scope: what
// the other SM's copies or warps wrote before is then ordered before what follows, the pair's MMAs among it (CTA scope was
// 0.3 us of 89 faster).
#pragma once

#include <cuda_fp16.h>

#include "merge.cuh"
#include "prefill_pair.cuh"

namespace hca {

struct PrefixParams {
    const int* seqlens;           // [B]
    const float* qscale;          // [B * Hq] logit scale (log2) of each row of the normalised queries, or null
    float* pfx_m;                 // [clusters + row tiles][256] references
    float* pfx_l;                 // sums of 2^(z - m)
    int B, Hq, Hkv, G, tpt, blk, W, Np, nct;
    long long total;              // pairs of the list
    int max_clusters, sms, cap;   // for shared_plan; own entries that a sequence's cache can hold
    float scale_log2;
};

// Consecutive key tiles j0 .. j0 + n - 1 of one row tile within a cluster's range (n = 0: no more).
struct PfxPiece {
    int rt, g, b0, j0, n;
    long long next;
};

__device__ __forceinline__ PfxPiece pfx_piece(const PrefixParams& p, long long x, long long end) {
    PfxPiece it = {};
    if (x >= end) return it;
    it.rt = (int)(x / p.nct);
    it.j0 = (int)(x % p.nct);
    it.n = (int)min((long long)(p.nct - it.j0), end - x);
    it.next = x + it.n;
    it.g = it.rt % p.Hkv;
    it.b0 = it.rt / p.Hkv * (2 * p.tpt);
    return it;
}
__device__ __forceinline__ int pfx_keys(const PrefixParams& p, const PfxPiece& it, int j) {
    return min(kPpKeys, p.Np - kPpKeys * (it.j0 + j));
}
// Tiles of 128 keys of a sequence's own entries and window (as q_keys_of and q_tiles of decode_quant.cuh count them).
__device__ __forceinline__ long long own_tiles(int L, int W, int blk, int Np, long long cap) {
    L = max(L, 1);
    const long long a = (long long)L - W, n0 = a > 0 ? a / blk : 0;
    const long long n = min(n0 > Np ? n0 - Np : 0, cap);
    return (n + kDecTile - 1) / kDecTile + (min(L, W) + kDecTile - 1) / kDecTile;
}
// Prefix entries visible to row r of an SM's half of the tile (= sequence * G + head); rows without a sequence see none.
__device__ __forceinline__ int pfx_visible(const PrefixParams& p, const PfxPiece& it, int half, int r) {
    const int b = it.b0 + half * p.tpt + r / p.G;
    if (r >= p.tpt * p.G || b >= p.B) return 0;
    const long long a = (long long)__ldg(p.seqlens + b) - p.W;
    return a > 0 ? (int)min((long long)p.Np, a / p.blk) : 0;
}

// Logit scale (log2) of that row's normalised query.
__device__ __forceinline__ float pfx_qscale(const PrefixParams& p, const PfxPiece& it, int half, int r) {
    const int b = it.b0 + half * p.tpt + r / p.G;
    return r < p.tpt * p.G && b < p.B ? __ldg(p.qscale + (size_t)b * p.Hq + it.g * p.G + r % p.G) : 0.f;
}

// MMA columns of a tile of nk keys: each SM of the pair holds half of them, in rows of 16
__device__ __forceinline__ int pfx_cols(int nk) { return (nk + 31) & ~31; }

// QK normalisation: one warp for two rows.  The keys become k / rms(k) and the queries q / rms(q) * g_q * g_k, both in
// fp16: normalised keys are at most sqrt(512), and a query is scaled by the power of two that puts its largest
// magnitude into [2^13, 2^14) (undone in its logit scale), so both fit, and are rounded to 11 bits where bf16 has
// 8 (with bf16 queries the outputs of 8191 entries were 1.7 times further off).
struct PrefixPrepParams {
    const __nv_bfloat16* q;       // [B * Hq][512]
    const __nv_bfloat16* kp;      // [Np * Hkv][512]
    const float* gq;
    const float* gk;
    __half* qn;                   // [B * Hq][512]
    __half* kn;                   // [Np * Hkv][512]
    float* qscale;                // [B * Hq]
    long long nq, nk;             // rows
    float eps, scale_log2;
};

constexpr int kPrepThreads = 256;
constexpr int kPrepRows = 2;      // rows per warp

__global__ void __launch_bounds__(kPrepThreads) prefix_prep_kernel(const PrefixPrepParams p) {
    // the prefix pass may set itself up meanwhile; it waits for this grid before it reads the rows
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long i0 = ((long long)blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5)) * kPrepRows;
    uint4 x[kPrepRows][2];
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k) {
        const long long i = i0 + k;
        if (i < p.nq + p.nk) {
            const uint4* src = reinterpret_cast<const uint4*>(i < p.nq ? p.q + i * kPpD : p.kp + (i - p.nq) * kPpD);
            x[k][0] = __ldg(src + lane);
            x[k][1] = __ldg(src + 32 + lane);
        }
    }
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k) {
        const long long i = i0 + k;
        if (i >= p.nq + p.nk) return;
        float f[16];
        float ss = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t w[4] = {x[k][u].x, x[k][u].y, x[k][u].z, x[k][u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[8 * u + 2 * e] = bf16lo(w[e]);
                f[8 * u + 2 * e + 1] = bf16hi(w[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        float inv = rsqrtf(ss * (1.f / kPpD) + p.eps);
        __half* dst = p.kn + (i - p.nq) * kPpD;
        if (i < p.nq) {
            float am = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const int c = 8 * (32 * u + lane) + e;
                    const float2 a = __ldg(reinterpret_cast<const float2*>(p.gq + c));
                    const float2 b = __ldg(reinterpret_cast<const float2*>(p.gk + c));
                    f[8 * u + e] *= inv * a.x * b.x;
                    f[8 * u + e + 1] *= inv * a.y * b.y;
                    am = fmaxf(am, fmaxf(fabsf(f[8 * u + e]), fabsf(f[8 * u + e + 1])));
                }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, off));
            // am = y * 2^(b - 127), 1 <= y < 2; factors in [2^-100, 2^100]
            const int b = min(max((int)(__float_as_uint(am) >> 23), 40), 240);
            inv = __uint_as_float((uint32_t)(267 - b) << 23);               // 2^(13 - (b - 127))
            if (lane == 0) p.qscale[i] = p.scale_log2 * __uint_as_float((uint32_t)(b - 13) << 23);
            dst = p.qn + i * kPpD;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __half2 h = __floats2half2_rn(f[8 * u + 2 * e] * inv, f[8 * u + 2 * e + 1] * inv);
                y[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            reinterpret_cast<uint4*>(dst)[32 * u + lane] = make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
}

// A row's reference moves when a logit exceeds it by this (log2).  P = 2^(z - m) is a floating number, so its
// relative precision does not depend on m; the bound only keeps sums of P v in range (|v| < 2^80), and is wide
// because a move costs a rescaling of O (thousands of cycles, against 6200 for a tile): with 2^8 and one key in a
// hundred 8 times larger, every second unit of 8191 entries moved.
constexpr float kPxRescale = 32.f;
constexpr int kPxRing = 6;                        // 16 KB slabs of K, or units of V, in flight per SM
constexpr uint32_t kPxSlab = 16384;               // K: 128 keys x 64 channels; V: 64 keys x 128 channels
// barriers: the S pair and the O pair use their own subsets of one numbering (the leaders are ranks 0 and 2)
enum : int {
    kPxFull = 0, kPxEmpty = 6,                    // slabs of both SMs landed (leader) / consumed (both)
    kPxSFull = 12, kPxSEmpty = 14,                // S tile ready (both) / read (leader)
    kPxPCons = 16,                                // P unit consumed: all four
    kPxPFull = 20, kPxCorr = 24,                  // P unit landed (each O rank) / checked and rescaled (leader)
    kPxOFull = 28, kPxOEmpty = 29, kPxDrain = 30,
    kPxQFull = 32, kPxQEmpty = 40,                // per Q slab: landed (leader) / free (both)
    kPxXch = 48                                   // maxima of an S tile exchanged, per TMEM lane quarter
};

__device__ __forceinline__ uint32_t px_idesc(int N, int b_mn) { return idesc_bf16(256, N, 0, b_mn); }
// both operands fp16
__device__ __forceinline__ uint32_t px_idesc_f16(int N) { return idesc_bf16(256, N, 0, 0) & ~((7u << 7) | (7u << 10)); }
__device__ __forceinline__ void px_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// Arrive on the barrier at this offset of every CTA in `mask` when the pair's MMAs issued so far have completed.
__device__ __forceinline__ void px_commit(uint64_t* bar, uint32_t mask) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(smem_u32(bar)), "h"((uint16_t)mask) : "memory");
}
// Arrival that orders no memory: what it announces is that this warp's tensor-memory loads are done (waited for
// before).  A release would also wait for the P stores in flight (1300 cycles a tile).
__device__ __forceinline__ void px_remote_arrive_relaxed(uint32_t rbar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(rbar) : "memory");
}
// Load into this CTA's shared memory, counted on a barrier of the pair's leader (a shared::cluster address).
__device__ __forceinline__ void px_load_4d(void* dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void px_tmem_alloc(uint32_t* dst) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(dst)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void px_tmem_dealloc(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(512) : "memory");
}
// A producer that gave up: its copies count on the leader's barrier, which it cannot wait on from here.  They take
// microseconds; give them a millisecond before this SM's memory is released.
__device__ __forceinline__ void px_settle() {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
}

template <bool NORM>
__global__ void __launch_bounds__(kPpThreads, 1)
prefix_kernel(const PrefixParams p, const __grid_constant__ CUtensorMap tm_q,
              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ CUtensorMap tm_out) {
    extern __shared__ __align__(1024) uint8_t dsmem[];
    uint8_t* sm = dsmem;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kPpSmBar);
    int* misc = reinterpret_cast<int*>(sm + kPpSmMisc);
    volatile int* abort_flag = misc;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = pp_cluster_rank();
    const bool s_cta = rank < 2;
    const int half = rank & 1;                    // this SM's 128 rows of the tile
    const bool leader = half == 0;
    // the swizzled operand tiles need a 1024-byte aligned base; there is no room for slack
    const bool aligned = (smem_u32(dsmem) & 1023u) == 0;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        misc[2] = aligned ? 1 : 0;
        for (int i = 0; i < kPxRing; ++i) {
            mbar_init(&bars[kPxFull + i], 1);
            mbar_init(&bars[kPxEmpty + i], 1);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&bars[kPxQFull + i], 1);
            mbar_init(&bars[kPxQEmpty + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[kPxSFull + i], 1);
            mbar_init(&bars[kPxSEmpty + i], 2 * kPpSoftWarps);
        }
        for (int i = 0; i < kPpSlots; ++i) {
            mbar_init(&bars[kPxPCons + i], 1);
            mbar_init(&bars[kPxPFull + i], 4);         // armed by each TMEM lane quarter
            mbar_init(&bars[kPxCorr + i], 8);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bars[kPxXch + i], 2);
        mbar_init(&bars[kPxOFull], 1);
        mbar_init(&bars[kPxOEmpty], 16);
        mbar_init(&bars[kPxDrain], 1);
        fence_mbar_init();
        if (s_cta) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
        } else {
            prefetch_tmap(&tm_v);
            prefetch_tmap(&tm_out);
        }
    }
    if (warp == 1) px_tmem_alloc(tmem_slot);
    // the own pass may start beside this one
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 2) {
        long long own = 0;
        for (int b = lane; b < p.B; b += 32) own += own_tiles(__ldg(p.seqlens + b), p.W, p.blk, p.Np, p.cap);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) own += __shfl_xor_sync(0xffffffffu, own, off);
        const SharedPlan plan = shared_plan_warp(p.total, own * p.Hkv, p.B * p.Hkv, p.max_clusters, p.sms);
        if (lane == 0) misc[3] = min((int)(gridDim.x >> 2), plan.clusters);
    }
    tc_fence_before();
    __syncthreads();
    pp_cluster_sync();      // every CTA's barriers are initialised before any remote arrive
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t peer_base = pp_mapa(smem_u32(sm), rank ^ 2u);          // S rank h <-> O rank h
    const uint32_t lead_bars = pp_mapa(smem_u32(bars), rank & 2u);        // barriers of the pair's leader
    const uint32_t pair_mask = s_cta ? 0x3u : 0xcu;
    bool go = true;
    for (uint32_t c = 0; c < 4; ++c) go &= pp_ld_cluster_u32(pp_mapa(smem_u32(misc + 2), c)) != 0;
    if (!go && threadIdx.x == 0) record_error(HCA_ERR_INTERNAL);
    if (NORM) asm volatile("griddepcontrol.wait;" ::: "memory");       // prefix_prep_kernel's rows
    const int cl = blockIdx.x >> 2;               // this cluster's range of the list of (row tile, key tile)
    const long long per = pfx_per(p.total, misc[3]);
    const long long x_beg = min(p.total, cl * per), x_end = min(p.total, x_beg + per);

    if (s_cta && warp == 0) {
        // ===================================================== S pair: TMA of Q and K
        if (lane == 0 && go) {
            uint32_t kr = 0, qn = 0;
            bool ok = true;
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end)) {
                for (int j = 0; ok && j < it.n; ++j) {
                    // the pair's N = 256 (or the 32-rounded key count) splits evenly over the two SMs
                    const int row = (it.j0 + j) * kPpKeys + half * (pfx_cols(pfx_keys(p, it, j)) / 2);
                    for (int s = 0; s < 8; ++s) {
                        if (j == 0) {
                            // Q slab s of this row tile, as soon as the previous row tile's last
                            // MMAs on slab s have completed (not after its whole last tile)
                            if (!pp_wait_cl(&bars[kPxQEmpty + s], (qn & 1) ^ 1, abort_flag)) {
                                ok = false;
                                break;
                            }
                            if (leader)
                                mbar_arrive_expect_tx(&bars[kPxQFull + s], 2u * (uint32_t)(p.tpt * p.G) * 128u);
                            px_load_4d(sm + kPpSmQ + s * kPpQSlab, &tm_q, lead_bars + (kPxQFull + s) * 8, 64 * s,
                                       it.g * p.G, it.b0 + half * p.tpt, 0);
                        }
                        const uint32_t st = kr % kPxRing;
                        if (!pp_wait_cl(&bars[kPxEmpty + st], ((kr / kPxRing) & 1) ^ 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        if (leader) mbar_arrive_expect_tx(&bars[kPxFull + st], 2 * kPxSlab);
                        px_load_4d(sm + kPpSmRing + st * kPxSlab, &tm_k, lead_bars + (kPxFull + st) * 8, 64 * s, it.g, row, 0);
                        ++kr;
                    }
                }
                ++qn;
            }
            if (!ok || *abort_flag) px_settle();
        }
    } else if (rank == 0 && warp == 1) {
        // ===================================================== S pair: S = Q K^T
        if (go) {
            uint32_t kr = 0;
            int n = 0, item_n = 0;
            bool ok = true;
            const uint32_t q_base = smem_u32(sm + kPpSmQ);
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end), ++item_n) {
                for (int j = 0; ok && j < it.n; ++j, ++n) {
                    const int sb = n & 1;
                    if (!pp_warp_wait_cl(&bars[kPxSEmpty + sb], ((n >> 1) & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int cols = pfx_cols(pfx_keys(p, it, j));
                    const uint32_t id = NORM ? px_idesc_f16(cols) : px_idesc(cols, 0);
                    const uint32_t dst = tmem + sb * kPpKeys;
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t st = kr % kPxRing;
                        // Q slab s of this row tile (landed once per item, used by every tile)
                        if ((j == 0 && !pp_warp_wait_cl(&bars[kPxQFull + s], item_n & 1, abort_flag)) ||
                            !pp_warp_wait_cl(&bars[kPxFull + st], (kr / kPxRing) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t kb = smem_u32(sm + kPpSmRing + st * kPxSlab);
                            const uint32_t qa = q_base + s * kPpQSlab;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                px_mma(dst, smem_desc_sw128(qa + kk * 32, 16, 1024),
                                       smem_desc_sw128(kb + kk * 32, 16, 1024), id, (s | kk) ? 1u : 0u);
                            px_commit(&bars[kPxEmpty + st], pair_mask);
                            // the row tile's last use of Q slab s: the next row tile's slab s
                            // may land once these MMAs have completed
                            if (j == it.n - 1) px_commit(&bars[kPxQEmpty + s], pair_mask);
                        }
                        __syncwarp();
                        ++kr;
                    }
                    if (!ok) break;
                    if (elect_one()) px_commit(&bars[kPxSFull + sb], pair_mask);
                    __syncwarp();
                }
            }
            if (elect_one()) {
                px_commit(&bars[kPxDrain], 1u << rank);
                pp_drain_wait(&bars[kPxDrain], 0);
            }
            __syncwarp();
        }
    } else if (s_cta && warp >= 2 && warp < 2 + kPpSoftWarps) {
        // ===================================================== S pair: softmax, P to the O pair
        // Eight warps: warp w owns the 32 rows of TMEM lane quarter w % 4 and one half of the
        // columns of every unit (hw = 0: the first 64, hw = 1: the last 64).  The two warps of
        // a quarter keep identical per-row references m (they take the same decisions from the same
        // exchanged maxima), and take them for a whole tile before its first store: stores of
        // st.async to one address land in no order, so a unit is not stored again.
        if (go) {
            const int q4 = warp & 3;
            const int hw = (warp - 2) >> 2;
            const int r = q4 * 32 + lane;
            const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
            const bool neg = p.scale_log2 < 0.f;                      // of a row's logits, the least is then the largest
            const int c0 = 64 * hw;                                   // this warp's columns of a unit
            float* xch = reinterpret_cast<float*>(sm + kPpSmXch);     // [2 parities][2 halves][128 rows]
            const uint32_t rP = peer_base + kPpSmP + (uint32_t)r * 16u + (uint32_t)hw * 16384u;
            const uint32_t rHdr = peer_base + kPpSmHdr;
            const uint32_t rPFull = peer_base + kPpSmBar + kPxPFull * 8;
            // S tile n, of whose columns this row sees the first `hi`: wait for it, and give the other warp of the quarter the
            // extreme logit over this warp's columns
            auto publish = [&](int n, int hi, int nu) {
                const uint32_t sa = tmem + lane_off + (n & 1) * kPpKeys + c0;
                float e0 = neg ? INFINITY : -INFINITY, e1 = e0;
#pragma unroll 1
                for (int hh = 0; hh < nu; ++hh) {
                    float v[32], w[32];
                    tmem_ld32(sa + hh * kPpUKeys, v);
                    tmem_ld32(sa + hh * kPpUKeys + 32, w);
                    tmem_wait_ld32(v);
                    tmem_wait_ld32(w);
                    const int lim = hi - hh * kPpUKeys - c0;
                    if (__all_sync(0xffffffffu, lim >= 64)) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            e0 = neg ? min3(e0, v[e], v[e + 1]) : max3(e0, v[e], v[e + 1]);
                            e1 = neg ? min3(e1, w[e], w[e + 1]) : max3(e1, w[e], w[e + 1]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (e < lim) e0 = neg ? fminf(e0, v[e]) : fmaxf(e0, v[e]);
                            if (e + 32 < lim) e1 = neg ? fminf(e1, w[e]) : fmaxf(e1, w[e]);
                        }
                    }
                }
                const float ext = neg ? fminf(e0, e1) : fmaxf(e0, e1);
                xch[((n & 1) * 2 + hw) * 128 + r] = ext;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kPxXch + q4]);
                return ext;
            };
            int n = 0;            // S tiles
            uint32_t un = 0;      // P units
            bool ok = true;
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end)) {
                const int vis = pfx_visible(p, it, half, r);        // prefix entries that this row sees
                const float sl2 = NORM ? pfx_qscale(p, it, half, r) : p.scale_log2;
                float m = -INFINITY;
                for (int j = 0; ok && j < it.n; ++j, ++n) {
                    const int sb = n & 1;
                    const int nk = pfx_keys(p, it, j);
                    const int key0 = (it.j0 + j) * kPpKeys;
                    const int hi = min(nk, vis - key0);           // valid columns of this row: [0, hi)
                    const int nu = pp_units(nk);
                    if (!pp_warp_wait_cl(&bars[kPxSFull + sb], (n >> 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float ext = publish(n, hi, nu);
                    if (!warp_wait(&bars[kPxXch + q4], n & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const float other = xch[(sb * 2 + (hw ^ 1)) * 128 + r];
                    // The reference maximum m of a row is lazy: P = 2^(logit - m) is computed against the reference of
                    // the earlier tiles, and m moves only when a tile exceeds it by kPxRescale (or the row had none).
                    const bool fresh = m == -INFINITY;
                    bool resc = false;
                    float al = 1.f;
                    const float dm = hi > 0 ? fmaf(neg ? fminf(ext, other) : fmaxf(ext, other), sl2, fresh ? 0.f : -m) : -INFINITY;
                    if (fresh ? dm > -INFINITY : dm > kPxRescale) {
                        const float mn = fresh ? dm : m + dm;
                        if (!fresh) {
                            al = ex2(m - mn);
                            resc = true;
                        }
                        m = mn;
                    }
                    const bool any = __any_sync(0xffffffffu, resc);
                    const float mref = m == -INFINITY ? 0.f : m;
                    const float2 sl = make_float2(sl2, sl2), nm = make_float2(-mref, -mref);
                    const uint32_t sa = tmem + lane_off + sb * kPpKeys + c0;
                    for (int hh = 0; hh < nu; ++hh, ++un) {
                        const int us = (int)(un % kPpSlots);
                        const int u_cols = pp_unit_cols(nk, hh) - c0;         // columns of this warp (none: <= 0)
                        const int lim = hi - hh * kPpUKeys - c0;              // valid ones of this row
                        // slot us of the O rank is free once the PV of unit un - kPpSlots has landed
                        if (!pp_warp_wait_cl(&bars[kPxPCons + us], ((un / kPpSlots) & 1) ^ 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        // P in bf16 straight into slot us of the O rank: keys 8c..8c+7 of the unit,
                        // this row, at chunk c (2 KB per chunk of 8 keys x 128 rows).  Every store
                        // counts its bytes on the slot's barrier, which each lane quarter arms below.
                        const uint32_t pbar = rPFull + us * 8;
                        const uint32_t pbase = rP + us * kPpPBuf;
                        // 16 columns from c
                        auto put16 = [&](auto masked_tag, const float* v, int c) {
                            constexpr bool kMasked = decltype(masked_tag)::value;
                            uint32_t pk[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float2 d = fma2(make_float2(v[2 * e], v[2 * e + 1]), sl, nm);
                                if (kMasked) {
                                    d.x = c + 2 * e < lim ? d.x : -INFINITY;
                                    d.y = c + 2 * e + 1 < lim ? d.y : -INFINITY;
                                }
                                pk[e] = pack_bf16x2(ex2(d.x), ex2(d.y));
                            }
                            const uint32_t ra = pbase + (uint32_t)c * 256u;
                            pp_st_async_v4(ra, pk[0], pk[1], pk[2], pk[3], pbar);
                            pp_st_async_v4(ra + 2048u, pk[4], pk[5], pk[6], pk[7], pbar);
                        };
                        const uint32_t su = sa + hh * kPpUKeys;
                        // columns valid for every row of the warp (most units) skip the per-column mask
                        if (__all_sync(0xffffffffu, lim >= 64)) {
                            // the second half's load runs while the first half is worked on
                            float v[32], w[32];
                            tmem_ld32(su, v);
                            tmem_wait_ld32(v);
                            tmem_ld32(su + 32, w);
                            put16(std::false_type{}, v, 0);
                            put16(std::false_type{}, v + 16, 16);
                            tmem_wait_ld32(w);
                            put16(std::false_type{}, w, 32);
                            put16(std::false_type{}, w + 16, 48);
                        } else {
#pragma unroll 1
                            for (int c = 0; c < min(u_cols, 64); c += 16) {
                                float v[16];
                                tmem_ld16(su + c, v);
                                tmem_wait_ld();
                                put16(std::true_type{}, v, c);
                            }
                        }
                        if (hh == nu - 1) {
                            // every TMEM load of this warp from the tile has completed
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) px_remote_arrive_relaxed(lead_bars + (kPxSEmpty + sb) * 8);
                        }
                        if (hw == 0) {
                            // unit header: rescale factor per row, per-quarter flag (a tile's first unit has both for the
                            // tile); then the arm: this quarter's P bytes (both warps) and header bytes
                            const uint32_t hdr = rHdr + us * kPpHdrBytes;
                            pp_st_async_u32(hdr + r * 4, __float_as_uint(hh ? 1.f : al), pbar);
                            if (lane == 0) {
                                pp_st_async_u32(hdr + 512 + q4 * 4, any && !hh ? 1u : 0u, pbar);
                                pp_remote_arrive_expect_tx(pbar, (uint32_t)u_cols * 64u + 32u * 4u + 4u);
                            }
                            if (j == it.n - 1 && hh == nu - 1)
                                p.pfx_m[(size_t)(cl + it.rt) * 256 + half * 128 + r] =
                                    vis > it.j0 * kPpKeys ? fmaxf(m, kLowest) : -INFINITY;
                        }
                    }
                }
            }
        }
    }
    else if (!s_cta && warp == 0) {
        // ===================================================== O pair: TMA of V
        if (lane == 0 && go) {
            uint32_t vr = 0;
            bool ok = true;
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end)) {
                for (int j = 0; ok && j < it.n; ++j) {
                    const int row = (it.j0 + j) * kPpKeys;
                    const int nk = pfx_keys(p, it, j);
                    for (int hh = 0; ok && hh < pp_units(nk); ++hh) {
                        const int nv = (pp_unit_keys(nk, hh) + 63) >> 6;
                        for (int h = 0; ok && h < 2; ++h)
                            for (int u = 0; u < nv; ++u) {
                                const uint32_t st = vr % kPxRing;
                                if (!pp_wait_cl(&bars[kPxEmpty + st], ((vr / kPxRing) & 1) ^ 1, abort_flag)) {
                                    ok = false;
                                    break;
                                }
                                if (leader) mbar_arrive_expect_tx(&bars[kPxFull + st], 2 * kPxSlab);
                                // this SM's half of the 256 value columns
                                for (int c = 0; c < 2; ++c)
                                    px_load_4d(sm + kPpSmVRing + st * kPxSlab + c * kPpVSub, &tm_v,
                                               lead_bars + (kPxFull + st) * 8, 256 * h + 128 * half + 64 * c, it.g,
                                               row + kPpUKeys * hh + 64 * u, 0);
                                ++vr;
                            }
                    }
                }
            }
            if (!ok || *abort_flag) px_settle();
        }
    } else if (rank == 2 && warp == 1) {
        // ===================================================== O pair: O += P V
        if (go) {
            uint32_t vr = 0, un = 0;
            int item_n = 0;
            bool ok = true;
            const uint32_t p_base = smem_u32(sm + kPpSmP);
            const uint32_t id = px_idesc(256, 1);
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end), ++item_n) {
                for (int j = 0; ok && j < it.n; ++j) {
                    const int nk = pfx_keys(p, it, j);
                    const int nu = pp_units(nk);
                    for (int hh = 0; hh < nu; ++hh, ++un) {
                        const int us = (int)(un % kPpSlots);
                        const uint32_t ph = (un / kPpSlots) & 1;
                        const bool first = j == 0 && hh == 0;
                        // both SMs' P has landed (seen, and handed to the async proxy, by their rescale warps) and
                        // their O rows are rescaled
                        if (!pp_warp_wait_cl(&bars[kPxCorr + us], ph, abort_flag) ||
                            (first && !pp_warp_wait_cl(&bars[kPxOEmpty], (item_n & 1) ^ 1, abort_flag))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const int nku = pp_unit_keys(nk, hh);
                        const int nv = (nku + 63) >> 6;
                        for (int h = 0; ok && h < 2; ++h)
                            for (int u = 0; u < nv; ++u) {
                                const uint32_t st = vr % kPxRing;
                                if (!pp_warp_wait_cl(&bars[kPxFull + st], (vr / kPxRing) & 1, abort_flag)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                if (elect_one()) {
                                    const uint32_t vb = smem_u32(sm + kPpSmVRing + st * kPxSlab);
                                    const uint32_t pa = p_base + us * kPpPBuf + u * 16384;   // 16 keys = 4 KB
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        if (64 * u + 16 * kk < nku)
                                            px_mma(tmem + 256 * h, pp_desc_noswz(pa + kk * 4096, 2048, 128),
                                                   smem_desc_sw128(vb + kk * 2048, kPpVSub, 1024), id,
                                                   (first && u == 0 && kk == 0) ? 0u : 1u);
                                    px_commit(&bars[kPxEmpty + st], pair_mask);
                                }
                                __syncwarp();
                                ++vr;
                            }
                        if (!ok) break;
                        if (elect_one()) {
                            px_commit(&bars[kPxPCons + us], 0xfu);
                            if (j == it.n - 1 && hh == nu - 1) px_commit(&bars[kPxOFull], pair_mask);
                        }
                        __syncwarp();
                    }
                }
            }
            if (elect_one()) {
                px_commit(&bars[kPxDrain], 1u << rank);
                pp_drain_wait(&bars[kPxDrain], 0);
            }
            __syncwarp();
        }
    } else if (!s_cta && warp >= 2) {
        // ===================================================== O pair: rescale (warps 2-5), epilogue (2-9)
        if (go) {
            const int q4 = warp & 3;
            const bool extra = warp > 5;            // shares the quarter's epilogue only
            const int r = q4 * 32 + lane;
            const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
            uint32_t un = 0;
            int item_n = 0;
            bool ok = true;
            // a quarter's two warps go on or unwind together
            auto pair_agree_o = [&](bool ok_mine) -> bool {
                uint32_t res;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                             "barrier.red.and.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(res) : "r"((uint32_t)ok_mine), "r"(8 + q4) : "memory");
                return res != 0;
            };
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end), ++item_n) {
                float l = 0.f;            // row sum of the bf16 P this CTA multiplies with
                for (int j = 0; !extra && ok && j < it.n; ++j) {
                    const int nk = pfx_keys(p, it, j);
                    const int nu = pp_units(nk);
                    for (int hh = 0; hh < nu; ++hh, ++un) {
                        const int us = (int)(un % kPpSlots);
                        if (!pp_warp_wait_cl(&bars[kPxPFull + us], (un / kPpSlots) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint8_t* hdr = sm + kPpSmHdr + us * kPpHdrBytes;
                        const int flag = *reinterpret_cast<const volatile int*>(hdr + 512 + q4 * 4);
                        const float al = *reinterpret_cast<const volatile float*>(hdr + r * 4);
                        // l = l * alpha + the unit's P of this row (8 keys per 16-byte chunk)
                        float us_sum = 0.f;
                        const uint8_t* prow = sm + kPpSmP + us * kPpPBuf + r * 16;
                        const int nch = pp_unit_cols(nk, hh) >> 3;
#pragma unroll 4
                        for (int c = 0; c < nch; ++c) {
                            const uint4 w = *reinterpret_cast<const uint4*>(prow + c * 2048);
                            us_sum += (bf16lo(w.x) + bf16hi(w.x)) + (bf16lo(w.y) + bf16hi(w.y)) +
                                      (bf16lo(w.z) + bf16hi(w.z)) + (bf16lo(w.w) + bf16hi(w.w));
                        }
                        l = l * al + us_sum;
                        if (flag) {
                            // a row of this warp moved its reference maximum (never in the first
                            // unit of an item): scale O once the PV of unit un-1 has landed
                            const uint32_t pu = un - 1;
                            if (!pp_warp_wait_cl(&bars[kPxPCons + pu % kPpSlots], (pu / kPpSlots) & 1, abort_flag)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int c0 = 0; c0 < kPpD; c0 += 32) {
                                float o[32];
#pragma unroll
                                for (int k = 0; k < 2; ++k) tmem_ld16(tmem + lane_off + c0 + 16 * k, o + 16 * k);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    uint32_t w[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[16 * k + e] * al);
                                    tmem_st16(tmem + lane_off + c0 + 16 * k, w);
                                }
                            }
                            tmem_wait_st();
                        }
                        fence_proxy_async_smem();     // P came through the generic proxy; the pair's MMAs read it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) pp_remote_arrive(lead_bars + (kPxCorr + us) * 8);
                    }
                }
                if (!pair_agree_o(ok)) break;
                // ---- epilogue: the record (l, O), half of the columns for each of a quarter's two warps.  Each warp stages 32 rows x 128 bytes at a time in
                // shared memory and writes them with one TMA tensor store (a coalesced box);
                // per-lane row stores would touch 32 lines per instruction.
                if (!pair_agree_o(pp_warp_wait_cl(&bars[kPxOFull], item_n & 1, abort_flag))) break;
                tc_fence_after();
                if (!extra) p.pfx_l[(size_t)(cl + it.rt) * 256 + half * 128 + r] = l;
                uint8_t* stg = sm + kPpSmStage + (q4 * 2 + extra) * (kPpStageWarp / 2);
                const int r0 = q4 * 32;                       // first row of this warp's box
                const int orow = (cl + it.rt) * 256 + half * 128 + r0;
#pragma unroll 1
                for (int c0 = extra * (kPpD / 2), k = 0; k < kPpD / 64; c0 += 32, ++k) {
                    float o[32];
                    tmem_ld16(tmem + lane_off + c0, o);
                    tmem_ld16(tmem + lane_off + c0 + 16, o + 16);
                    tmem_wait_ld();
                    if (lane == 0) pp_bulk_wait_read0();              // the previous piece's store has read it
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e)       // 128-byte swizzle: chunk e of row lane
                        *reinterpret_cast<float4*>(stg + lane * 128 + (((e ^ lane) & 7) << 4)) =
                            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        pp_tma_store_4d(&tm_out, stg, c0, orow, 0, 0);
                        pp_bulk_commit();
                    }
                }
                if (lane == 0) pp_bulk_wait_read0();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pp_remote_arrive(lead_bars + kPxOEmpty * 8);
            }
            if (lane == 0) pp_bulk_wait_all();     // every output store has completed
            __syncwarp();
        }
    }

    __syncwarp();           // every role reconverges its warp before the CTA-wide barrier
    tc_fence_before();
    __syncthreads();
    pp_cluster_sync();      // no remote store or arrive is still aimed at a CTA that leaves
    if (warp == 1) {
        tc_fence_after();
        px_tmem_dealloc(tmem);
    }
}

}  // namespace hca
