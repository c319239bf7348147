// prefix.cuh -- attention of a batch's queries to the entries that all its sequences share
// (first pass of hca_decode_shared).
//
// A common prefix of Np entries is held once.  The 64 heads of one sequence fill half an MMA tile and read every
// entry; here two sequences' heads (or tpt = 128 / G of them) stand in one tile of 128 rows, and every entry
// is read from L2 once per row tile instead of from memory once per sequence:
//   z[r, j] = scale q_r . k_j   over the entries j < min(Np, n_c) that row r's sequence sees,
// one softmax per row over a range of key tiles, kept as a record (m = log2 sum 2^z, O / l) that merge.cuh joins
// with the row's own entries and window.
//
// The list of (row tile, key tile of 256 entries) pairs, row tile by row tile, is cut into one range per
// cluster.  A cluster of two SMs shares the work by stage, as prefill_pair.cuh does (S = Q K^T and softmax on
// the first, O += P V with all 512 value columns in tensor memory on the second) and with its shared-memory
// layout and barriers.
#pragma once

#include "prefill_pair.cuh"

namespace hca {

struct PrefixParams {
    const int* seqlens;           // [B]
    const float* kinv;            // [Hkv][kstride] 1 / rms of the prefix keys (QK normalisation)
    float* pfx_m;                 // [clusters + row tiles][128]
    int B, Hq, Hkv, G, tpt, blk, W, Np, nct, kstride;
    long long total, per;         // pairs of the list, and of a cluster's range
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
    it.b0 = it.rt / p.Hkv * p.tpt;
    return it;
}
__device__ __forceinline__ int pfx_keys(const PrefixParams& p, const PfxPiece& it, int j) {
    return min(kPpKeys, p.Np - kPpKeys * (it.j0 + j));
}
// Prefix entries visible to row r (= sequence in the tile * G + head); rows without a sequence see none.
__device__ __forceinline__ int pfx_visible(const PrefixParams& p, const PfxPiece& it, int r) {
    const int b = it.b0 + r / p.G;
    if (r >= p.tpt * p.G || b >= p.B) return 0;
    const long long a = (long long)__ldg(p.seqlens + b) - p.W;
    return a > 0 ? (int)min((long long)p.Np, a / p.blk) : 0;
}

// QK normalisation: one warp per row.  Rows of q become q / rms(q) * g_q * g_k in bf16 (the keys then need only
// 1 / rms(k), which goes to kinv).
struct PrefixPrepParams {
    const __nv_bfloat16* q;       // [B * Hq][512]
    const __nv_bfloat16* kp;      // [Np][Hkv][512]
    const float* gq;
    const float* gk;
    __nv_bfloat16* qn;            // [B * Hq][512]
    float* kinv;                  // [Hkv][kstride]
    long long nq;                 // B * Hq
    int Np, Hkv, kstride;
    float eps;
};

constexpr int kPrepThreads = 256;

__global__ void __launch_bounds__(kPrepThreads) prefix_prep_kernel(const PrefixPrepParams p) {
    const int lane = threadIdx.x & 31;
    const long long nk = (long long)p.Np * p.Hkv;
    const long long i = (long long)blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
    if (i >= p.nq + nk) return;
    const bool isq = i < p.nq;
    const __nv_bfloat16* src = isq ? p.q + i * kPpD : p.kp + (i - p.nq) * kPpD;
    uint4 x[2];
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        x[u] = __ldg(reinterpret_cast<const uint4*>(src) + 32 * u + lane);
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(bf16lo(w[e]), bf16lo(w[e]), fmaf(bf16hi(w[e]), bf16hi(w[e]), ss));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float inv = rsqrtf(ss * (1.f / kPpD) + p.eps);
    if (!isq) {
        const long long r = i - p.nq;
        if (lane == 0) p.kinv[(r % p.Hkv) * p.kstride + r / p.Hkv] = inv;
        return;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int c = 8 * (32 * u + lane);
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 a = __ldg(reinterpret_cast<const float2*>(p.gq + c) + e), b = __ldg(reinterpret_cast<const float2*>(p.gk + c) + e);
            y[e] = pack_bf16x2(bf16lo(w[e]) * (inv * a.x * b.x), bf16hi(w[e]) * (inv * a.y * b.y));
        }
        reinterpret_cast<uint4*>(p.qn + i * kPpD)[32 * u + lane] = make_uint4(y[0], y[1], y[2], y[3]);
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
    const bool s_cta = rank == 0;
    // the swizzled operand tiles need a 1024-byte aligned base; there is no room for slack
    const bool aligned = (smem_u32(dsmem) & 1023u) == 0;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        misc[2] = aligned ? 1 : 0;
        for (int i = 0; i < kPpRingK; ++i) {
            mbar_init(&bars[kBarKFull + i], 1);
            mbar_init(&bars[kBarKEmpty + i], 1);
        }
        for (int i = 0; i < kPpRingV; ++i) {
            mbar_init(&bars[kBarVFull + i], 1);
            mbar_init(&bars[kBarVEmpty + i], 1);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&bars[kBarQSFull + i], 1);
            mbar_init(&bars[kBarQSEmpty + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[kBarSFull + i], 1);
            mbar_init(&bars[kBarSEmpty + i], kPpSoftWarps);
        }
        for (int i = 0; i < kPpSlots; ++i) {
            mbar_init(&bars[kBarPEmpty + i], 1);
            mbar_init(&bars[kBarPFull + i], 4);        // armed by each TMEM lane quarter
            mbar_init(&bars[kBarCorr + i], 4);
            mbar_init(&bars[kBarPCons + i], 1);
        }
        mbar_init(&bars[kBarOFull], 1);
        mbar_init(&bars[kBarOEmpty], 4);
        mbar_init(&bars[kBarDrain], 1);
        fence_mbar_init();
        if (s_cta) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
        } else {
            prefetch_tmap(&tm_v);
            prefetch_tmap(&tm_out);
        }
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    pp_cluster_sync();      // barriers of both CTAs are initialised before any remote arrive
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t peer_base = pp_mapa(smem_u32(sm), rank ^ 1u);
    const bool go = aligned && pp_ld_cluster_u32(peer_base + kPpSmMisc + 8) != 0;
    if (!go && threadIdx.x == 0) record_error(HCA_ERR_INTERNAL);
    const int cl = blockIdx.x >> 1;               // this cluster's range of the list of (row tile, key tile)
    const long long x_beg = cl * p.per, x_end = min(p.total, x_beg + p.per);

    if (s_cta && warp == 0) {
        // ===================================================== S-CTA: TMA of Q and K
        if (lane == 0 && go) {
            uint32_t kr = 0, qn = 0;
            bool ok = true;
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end)) {
                for (int j = 0; ok && j < it.n; ++j) {
                    const int row = (it.j0 + j) * kPpKeys;
                    for (int s = 0; s < 8; ++s) {
                        if (j == 0) {
                            // Q slab s of this row tile, as soon as the previous row tile's last
                            // MMAs on slab s have completed (not after its whole last tile)
                            if (!mbar_wait(&bars[kBarQSEmpty + s], (qn & 1) ^ 1, abort_flag)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(&bars[kBarQSFull + s], (uint32_t)(p.tpt * p.G) * 128u);
                            tma_load_4d(sm + kPpSmQ + s * kPpQSlab, &tm_q, &bars[kBarQSFull + s], 64 * s,
                                        it.g * p.G, it.b0, 0);
                        }
                        const uint32_t st = kr % kPpRingK;
                        if (!mbar_wait(&bars[kBarKEmpty + st], ((kr / kPpRingK) & 1) ^ 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&bars[kBarKFull + st], kPpUnit);
                        tma_load_4d(sm + kPpSmRing + st * kPpUnit, &tm_k, &bars[kBarKFull + st],
                                    64 * s, it.g, row, 0);
                        ++kr;
                    }
                }
                ++qn;
            }
            pp_drain_ring(&bars[kBarKFull], kr, kPpRingK);
            if (qn)
                for (int s = 0; s < 8; ++s) pp_drain_wait(&bars[kBarQSFull + s], (qn - 1) & 1);
        }
    } else if (s_cta && warp == 1) {
        // ===================================================== S-CTA: S = Q K^T
        if (go) {
            uint32_t kr = 0;
            int n = 0, item_n = 0;
            bool ok = true;
            const uint32_t q_base = smem_u32(sm + kPpSmQ);
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end), ++item_n) {
                for (int j = 0; ok && j < it.n; ++j, ++n) {
                    const int sb = n & 1;
                    if (!warp_wait(&bars[kBarSEmpty + sb], ((n >> 1) & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int N = (pfx_keys(p, it, j) + 15) & ~15;
                    const uint32_t id = idesc_bf16(128, N, 0, 0);
                    const uint32_t dst = tmem + sb * kPpKeys;
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t st = kr % kPpRingK;
                        // Q slab s of this row tile (landed once per item, used by every tile)
                        if ((j == 0 && !warp_wait(&bars[kBarQSFull + s], item_n & 1, abort_flag)) ||
                            !warp_wait(&bars[kBarKFull + st], (kr / kPpRingK) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (lane == 0) {
                            const uint32_t kb = smem_u32(sm + kPpSmRing + st * kPpUnit);
                            const uint32_t qa = q_base + s * kPpQSlab;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ss(dst, smem_desc_sw128(qa + kk * 32, 16, 1024),
                                       smem_desc_sw128(kb + kk * 32, 16, 1024), id, (s | kk) ? 1u : 0u);
                            mma_commit(&bars[kBarKEmpty + st]);
                            // the row tile's last use of Q slab s: the next row tile's slab s
                            // may land once these MMAs have completed
                            if (j == it.n - 1) mma_commit(&bars[kBarQSEmpty + s]);
                        }
                        __syncwarp();
                        ++kr;
                    }
                    if (!ok) break;
                    if (lane == 0) mma_commit(&bars[kBarSFull + sb]);
                    __syncwarp();
                }
            }
            if (lane == 0) {
                mma_commit(&bars[kBarDrain]);
                pp_drain_wait(&bars[kBarDrain], 0);
            }
            __syncwarp();
        }
    } else if (s_cta && warp >= 2 && warp < 2 + kPpSoftWarps) {
        // ===================================================== S-CTA: softmax, P to the O-CTA
        // Eight warps: warp w owns the 32 rows of TMEM lane quarter w % 4 and one half of the
        // columns of every unit (hw = 0: the first 64, hw = 1: the last 64).  The two warps of
        // a quarter keep identical per-row references m (they take the same decisions from
        // the same exchanged maxima) and their own partial row sums.
        if (go) {
            const int q4 = warp & 3;
            const int hw = (warp - 2) >> 2;
            const int r = q4 * 32 + lane;
            const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
            float* xch = reinterpret_cast<float*>(sm + kPpSmXch);     // [2 parities][2 halves][128 rows]
            int xpar = 0;
            // a value of this row from both warps of the quarter (64-thread named barrier)
            auto exchange = [&](float mine, float* other) {
                xch[(xpar * 2 + hw) * 128 + r] = mine;
                asm volatile("bar.sync %0, 64;" :: "r"(4 + q4) : "memory");
                *other = xch[(xpar * 2 + (hw ^ 1)) * 128 + r];
                xpar ^= 1;
            };
            // the two warps of a quarter go on or unwind together: a verdict that differed
            // would leave one of them at a named barrier the other never reaches
            auto pair_agree = [&](bool ok_mine) -> bool {
                uint32_t res;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                             "barrier.red.and.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(res) : "r"((uint32_t)ok_mine), "r"(4 + q4) : "memory");
                return res != 0;
            };
            const uint32_t rP = peer_base + kPpSmP + (uint32_t)r * 16u;
            const uint32_t rHdr = peer_base + kPpSmHdr;
            const uint32_t rPFull = peer_base + kPpSmBar + kBarPFull * 8;
            const float sl2 = p.scale_log2;
            int n = 0;            // S tiles
            uint32_t un = 0;      // P units
            bool ok = true;
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end)) {
                const int vis = pfx_visible(p, it, r);        // prefix entries that this row sees
                float m = -INFINITY, l = 0.f;     // l: this warp's partial row sum
                for (int j = 0; ok && j < it.n; ++j, ++n) {
                    const int sb = n & 1;
                    const int nk = pfx_keys(p, it, j);
                    const int key0 = (it.j0 + j) * kPpKeys;
                    const int hi = min(nk, vis - key0);           // valid columns of this row: [0, hi)
                    if (!pair_agree(warp_wait(&bars[kBarSFull + sb], (n >> 1) & 1, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = tmem + lane_off + sb * kPpKeys;
                    const float* kn = NORM ? p.kinv + (size_t)it.g * p.kstride + key0 : nullptr;   // 1 / rms of the keys
                    const int nu = pp_units(nk);
                    for (int hh = 0; hh < nu; ++hh, ++un) {
                        const int us = (int)(un % kPpSlots);
                        const int u_end = hh * kPpUKeys + pp_unit_cols(nk, hh);
                        const int c_beg = hh * kPpUKeys + 64 * hw;            // this warp's columns
                        const int c_end = min(c_beg + 64, u_end);             // (may be empty)
                        // The reference maximum m of a row is lazy: P = 2^(logit - m) is computed
                        // against the reference of the earlier units, and m moves only when a unit
                        // exceeds it by 2^8 -- the unit is then redone against the new reference.
                        // A quarter in which some row has no reference yet takes the maximum first.
                        const bool need_max = __any_sync(0xffffffffu, m == -INFINITY && hi > hh * kPpUKeys);
                        bool resc = false;
                        float al = 1.f;
                        if (need_max) {
                            float tmax = -INFINITY;
#pragma unroll 1
                            for (int c0 = c_beg; c0 < c_end; c0 += 32) {
                                float v[32];
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    if (c0 + 16 * k < c_end) tmem_ld16(sa + c0 + 16 * k, v + 16 * k);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const int c = c0 + k;
                                    if (c < hi) tmax = fmaxf(tmax, v[k] * (NORM ? sl2 * kn[c] : sl2));
                                }
                            }
                            float tother;
                            exchange(tmax, &tother);
                            tmax = fmaxf(tmax, tother);
                            resc = m != -INFINITY && tmax > m + kPfRescale;
                            if (resc) {
                                al = ex2(m - tmax);
                                l *= al;
                            }
                            if (resc || (m == -INFINITY && tmax > -INFINITY)) m = tmax;
                        }
                        // the O-CTA's slot us is free once the PV of unit un - kPpSlots has landed
                        if (!pair_agree(pp_warp_wait_cl(&bars[kBarPEmpty + us], ((un / kPpSlots) & 1) ^ 1,
                                                        abort_flag))) {
                            ok = false;
                            break;
                        }
                        // P in bf16 straight into the O-CTA's slot us: keys 8c..8c+7 of the unit,
                        // this row, at chunk c (2 KB per chunk of 8 keys x 128 rows).  Every store
                        // counts its bytes on the slot's barrier; each lane quarter arms it once
                        // it knows how many bytes it stored (a redone unit is stored twice).
                        const uint32_t pbar = rPFull + us * 8;
                        const uint32_t pbase = rP + us * kPpPBuf;
                        int attempts = 1;
                        // columns valid for every row of the warp (most compressed units) skip
                        // the per-column mask
                        const bool unmasked = __all_sync(0xffffffffu, hi >= c_end);
                        float rs, dmax;
                        auto pass2 = [&](auto masked_tag, float mref) {
                            constexpr bool kMasked = decltype(masked_tag)::value;
                            dmax = -INFINITY;
                            rs = 0.f;
#pragma unroll 1
                            for (int c0 = c_beg; c0 < c_end; c0 += 32) {
                                float v[32];
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    if (c0 + 16 * k < c_end) tmem_ld16(sa + c0 + 16 * k, v + 16 * k);
                                tmem_wait_ld();
#pragma unroll
                                for (int k16 = 0; k16 < 2; ++k16) {
                                    const int cb = c0 + 16 * k16;
                                    if (cb < c_end) {
                                        uint32_t pk[8];
#pragma unroll
                                        for (int e = 0; e < 8; ++e) {
                                            const int c = cb + 2 * e;
                                            float d0 = fmaf(v[16 * k16 + 2 * e], NORM ? sl2 * kn[c] : sl2, -mref);
                                            float d1 = fmaf(v[16 * k16 + 2 * e + 1], NORM ? sl2 * kn[c + 1] : sl2, -mref);
                                            if (kMasked) {
                                                d0 = c < hi ? d0 : -INFINITY;
                                                d1 = c + 1 < hi ? d1 : -INFINITY;
                                            }
                                            dmax = fmaxf(dmax, fmaxf(d0, d1));
                                            const float a = ex2(d0), b2 = ex2(d1);
                                            rs += a + b2;
                                            pk[e] = pack_bf16x2(a, b2);
                                        }
                                        const uint32_t ra = pbase + ((uint32_t)(cb - hh * kPpUKeys) >> 3) * 2048u;
                                        pp_st_async_v4(ra, pk[0], pk[1], pk[2], pk[3], pbar);
                                        pp_st_async_v4(ra + 2048u, pk[4], pk[5], pk[6], pk[7], pbar);
                                    }
                                }
                            }
                        };
                        for (int attempt = 0;; ++attempt) {
                            const float mref = m == -INFINITY ? 0.f : m;
                            if (unmasked)
                                pass2(std::false_type{}, mref);
                            else
                                pass2(std::true_type{}, mref);
                            if (need_max || attempt) break;
                            // every row has a reference here; redo if a unit exceeded it
                            float dother;
                            exchange(dmax, &dother);
                            dmax = fmaxf(dmax, dother);
                            const bool over = dmax > kPfRescale;
                            if (!__any_sync(0xffffffffu, over)) break;
                            if (over) {
                                al = ex2(-dmax);
                                l *= al;
                                m += dmax;
                                resc = true;
                            }
                            attempts = 2;
                        }
                        l += rs;
                        if (hh == nu - 1) {
                            // every TMEM load of this warp from the tile has completed
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars[kBarSEmpty + sb]);
                        }
                        const bool last = j == it.n - 1 && hh == nu - 1;
                        float lrow = 0.f;
                        if (last) {      // whole-row sums for the epilogue and the LSE
                            float lother;
                            exchange(l, &lother);
                            lrow = l + lother;
                        }
                        if (hw == 0) {
                            // unit header: rescale factor per row, per-quarter flag; then the arm:
                            // this quarter's P bytes (both warps, every attempt) and header bytes
                            const uint32_t hdr = rHdr + us * kPpHdrBytes;
                            pp_st_async_u32(hdr + r * 4, __float_as_uint(al), pbar);
                            const bool any = __any_sync(0xffffffffu, resc);
                            if (lane == 0) {
                                pp_st_async_u32(hdr + 512 + q4 * 4, any ? 1u : 0u, pbar);
                                pp_remote_arrive_expect_tx(
                                    pbar, (uint32_t)attempts * (uint32_t)(u_end - hh * kPpUKeys) * 64u + 32u * 4u + 4u);
                            }
                            if (last) p.pfx_m[(size_t)(cl + it.rt) * 128 + r] = m + log2f(lrow);
                        }
                    }
                }
            }
        }
    }
    else if (!s_cta && warp == 0) {
        // ===================================================== O-CTA: TMA of V
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
                                const uint32_t st = vr % kPpRingV;
                                if (!mbar_wait(&bars[kBarVEmpty + st], ((vr / kPpRingV) & 1) ^ 1, abort_flag)) {
                                    ok = false;
                                    break;
                                }
                                mbar_arrive_expect_tx(&bars[kBarVFull + st], kPpUnit);
                                for (int c = 0; c < 4; ++c)
                                    tma_load_4d(sm + kPpSmVRing + st * kPpUnit + c * kPpVSub, &tm_v,
                                                &bars[kBarVFull + st], 256 * h + 64 * c, it.g,
                                                row + kPpUKeys * hh + 64 * u, 0);
                                ++vr;
                            }
                    }
                }
            }
            pp_drain_ring(&bars[kBarVFull], vr, kPpRingV);
        }
    } else if (!s_cta && warp == 1) {
        // ===================================================== O-CTA: O += P V
        if (go) {
            uint32_t vr = 0, un = 0;
            int item_n = 0;
            bool ok = true;
            const uint32_t p_base = smem_u32(sm + kPpSmP);
            const uint32_t id = idesc_bf16(128, 256, 0, 1);
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end), ++item_n) {
                for (int j = 0; ok && j < it.n; ++j) {
                    const int nk = pfx_keys(p, it, j);
                    const int nu = pp_units(nk);
                    for (int hh = 0; hh < nu; ++hh, ++un) {
                        const int us = (int)(un % kPpSlots);
                        const uint32_t ph = (un / kPpSlots) & 1;
                        const bool first = j == 0 && hh == 0;
                        if (!pp_warp_wait_cl(&bars[kBarPFull + us], ph, abort_flag) ||
                            !warp_wait(&bars[kBarCorr + us], ph, abort_flag) ||
                            (first && !warp_wait(&bars[kBarOEmpty], (item_n & 1) ^ 1, abort_flag))) {
                            ok = false;
                            break;
                        }
                        fence_proxy_async_smem();    // P arrived through the generic proxy
                        tc_fence_after();
                        const int nku = pp_unit_keys(nk, hh);
                        const int nv = (nku + 63) >> 6;
                        for (int h = 0; ok && h < 2; ++h)
                            for (int u = 0; u < nv; ++u) {
                                const uint32_t st = vr % kPpRingV;
                                if (!warp_wait(&bars[kBarVFull + st], (vr / kPpRingV) & 1, abort_flag)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                if (lane == 0) {
                                    const uint32_t vb = smem_u32(sm + kPpSmVRing + st * kPpUnit);
                                    const uint32_t pa = p_base + us * kPpPBuf + u * 16384;   // 16 keys = 4 KB
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        if (64 * u + 16 * kk < nku)
                                            mma_ss(tmem + 256 * h, pp_desc_noswz(pa + kk * 4096, 2048, 128),
                                                   smem_desc_sw128(vb + kk * 2048, kPpVSub, 1024), id,
                                                   (first && u == 0 && kk == 0) ? 0u : 1u);
                                    mma_commit(&bars[kBarVEmpty + st]);
                                }
                                __syncwarp();
                                ++vr;
                            }
                        if (!ok) break;
                        if (lane == 0) {
                            mma_commit(&bars[kBarPCons + us]);
                            if (j == it.n - 1 && hh == nu - 1) mma_commit(&bars[kBarOFull]);
                        }
                        __syncwarp();
                    }
                }
            }
            if (lane == 0) {
                mma_commit(&bars[kBarDrain]);
                pp_drain_wait(&bars[kBarDrain], 0);
            }
            __syncwarp();
        }
    } else if (!s_cta && warp >= 2 && warp <= 5) {
        // ===================================================== O-CTA: rescale, epilogue
        if (go) {
            const int q4 = warp & 3;
            const int r = q4 * 32 + lane;
            const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
            uint32_t un = 0;
            int item_n = 0;
            bool ok = true;
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end), ++item_n) {
                float l = 0.f;            // row sum of the bf16 P this CTA multiplies with
                for (int j = 0; ok && j < it.n; ++j) {
                    const int nk = pfx_keys(p, it, j);
                    const int nu = pp_units(nk);
                    for (int hh = 0; hh < nu; ++hh, ++un) {
                        const int us = (int)(un % kPpSlots);
                        if (!pp_warp_wait_cl(&bars[kBarPFull + us], (un / kPpSlots) & 1, abort_flag)) {
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
                            if (!warp_wait(&bars[kBarPCons + pu % kPpSlots], (pu / kPpSlots) & 1, abort_flag)) {
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
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars[kBarCorr + us]);
                    }
                }
                if (!ok) break;
                // ---- epilogue: the record O / l.  Each warp stages 32 rows x 128 bytes at a time in
                // shared memory and writes them with one TMA tensor store (a coalesced box);
                // per-lane row stores would touch 32 lines per instruction.
                if (!warp_wait(&bars[kBarOFull], item_n & 1, abort_flag)) break;
                tc_fence_after();
                const float inv = l == 0.f ? 0.f : 1.f / l;       // a row that sees nothing here: zeros
                uint8_t* stg = sm + kPpSmStage + q4 * kPpStageWarp;
                const int r0 = q4 * 32;                       // first row of this warp's box
                const int orow = (cl + it.rt) * 128 + r0;
#pragma unroll 1
                for (int c0 = 0, k = 0; c0 < kPpD; c0 += 32, ++k) {
                    uint8_t* buf = stg + (k & 1) * (kPpStageWarp / 2);
                    if (k >= 2 && lane == 0) pp_bulk_wait_read1();     // the store of piece k-2 read it
                    __syncwarp();
                    float o[32];
                    tmem_ld16(tmem + lane_off + c0, o);
                    tmem_ld16(tmem + lane_off + c0 + 16, o + 16);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)       // 128-byte swizzle: chunk e of row lane
                        *reinterpret_cast<float4*>(buf + lane * 128 + (((e ^ lane) & 7) << 4)) =
                            make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        pp_tma_store_4d(&tm_out, buf, c0, orow, 0, 0);
                        pp_bulk_commit();
                    }
                }
                if (lane == 0) pp_bulk_wait_read0();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kBarOEmpty]);
            }
            if (lane == 0) pp_bulk_wait_all();     // every output store has completed
            __syncwarp();
        }
    } else if (!s_cta && warp == 7) {
        // ===================================================== O-CTA: P slot consumed -> S-CTA
        if (lane == 0 && go) {
            const uint32_t rPEmpty = peer_base + kPpSmBar + kBarPEmpty * 8;
            uint32_t un = 0;
            bool ok = true;
            for (PfxPiece it = pfx_piece(p, x_beg, x_end); ok && it.n; it = pfx_piece(p, it.next, x_end)) {
                for (int j = 0; ok && j < it.n; ++j) {
                    const int nu = pp_units(pfx_keys(p, it, j));
                    for (int hh = 0; hh < nu; ++hh, ++un) {
                        const int us = (int)(un % kPpSlots);
                        if (!mbar_wait(&bars[kBarPCons + us], (un / kPpSlots) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        pp_remote_arrive(rPEmpty + us * 8);
                    }
                }
            }
        }
    }

    __syncwarp();           // every role reconverges its warp before the CTA-wide barrier
    tc_fence_before();
    __syncthreads();
    pp_cluster_sync();      // no remote store or arrive is still aimed at a CTA that leaves
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace hca
