// decode_quant.cuh -- split-KV HCA decode over an 8-bit compressed cache (hca_decode_quant).
//
// Same operation and work decomposition as decode.cuh (one query per sequence over its entries and its
// raw window, the batch's key tiles cut into one range per CTA, partial records merged afterwards); the
// entries are e4m3 codes with one power-of-two scale per key and per value vector (fp8.cuh), the window
// is raw bf16.  Entries go from memory to the tensor cores as they are (kind::f8f6f4, K = 32): widening
// them on the way would cost more shared-memory bandwidth than HBM delivers bytes (write 64 KB, read 64 KB,
// write 128 KB, read 128 KB per 128 keys of K and again of V).  The other operands are bf16 quantities, so
// each is split into two 8-bit terms, both multiplied with the same 8-bit tile into one fp32 accumulator:
//   q = hi + lo, both e4m3, after a power-of-two scale per head that puts max|q| in (224, 448].  hi keeps 4
//       significant bits and lo the next 4: a bf16 query (8 bits) is represented exactly down to 2^-10 of its
//       head's largest channel, and to 2^-18.8 of that channel below.  Same rounding (2^-8 at most) as bf16
//       for the fp32 queries that QK normalisation makes.
//   p = hi (e4m3) + lo (e5m2): where hi is normal (p >= 2^-6, 2^-12 of the row's largest) at most 2^-4 * 2^-3 =
//       2^-7 off, 2^-10 in the mean square; below, hi is within 2^-10 and lo within 2^-3 of the rest: 2^-13, or
//       2^-19 of the largest.  lo is e5m2 because its range matters more than its last bit: a probability down to
//       2^-22 of the largest still has a term, so a long tail of small probabilities is kept.
// The scale of a value vector belongs to the key, which is the contraction's axis, so it goes into p: with
// y = z + log2(vscale), the accumulators hold sums of 2^(y - m) * code, the reference m is the running
// maximum of y, and the row sum l adds 2^(y - m) / vscale = 2^(z - m).  m is kept 2^6 below the maximum
// and moves when some y exceeds it by 2^8, so that p <= 256 and 2^6 for the largest key: e4m3 ends at 448.
//
// Inside a CTA (12 warps: a thirteenth would leave 128 registers per thread instead of 168):
//   warp 0, 3   TMA of K / of V: slabs of 16 KB (128 keys x 128 codes, or x 64 bf16 channels of the window)
//               through a ring of four each; a tile of entries fills a ring once, a window tile twice;
//   warp 1      TMA of the query rows, once per (unit, kind of tile): 8-bit hi / lo for entries (made in place
//               by the softmax warps), bf16 for the window;  tcgen05.mma  S^T[128 keys x 64 heads] = K Q^T;
//   warp 2      tcgen05.mma  O^T[512 x 64] += V^T P^T;
//   warps 4-11  softmax, two per TMEM lane quarter, thread = (key row, 32 heads); record at a piece's end.
#pragma once

#include "decode.cuh"
#include "fp8.cuh"
#include "merge.cuh"

namespace hca {

constexpr int kQdThreads = 384;
constexpr int kQdSoftWarp0 = 4;
constexpr int kQdRing = 4;                 // slabs per ring (K, V)
constexpr int kQdLook = 4;                 // S buffers (2 with QK normalisation)
constexpr int kQdLookNorm = 2;
constexpr float kQdShift = 6.0f;           // the reference m lies this far (log2) below the maximum

constexpr uint32_t kQsQ = 0;
constexpr uint32_t kQsP = kQsQ + kDecQBytes;
constexpr uint32_t kQsK = kQsP + kDecPBufs * kDecPBytes;
constexpr uint32_t kQsV = kQsK + kQdRing * kSlabBytes;
constexpr uint32_t kQsBar = kQsV + kQdRing * kSlabBytes;
constexpr int kQdBars = 4 * kQdRing + 3 + 2 * kQdLook + 2 * kDecPBufs + 2;
constexpr uint32_t kQsRed = (kQsBar + kQdBars * 8 + 127) & ~127u;   // float[4][64]
constexpr uint32_t kQsMax = kQsRed + 4 * 64 * 4;                    // float[64] reference m per head
constexpr uint32_t kQsAlpha = kQsMax + 64 * 4;                      // float[64] rescale factors
constexpr uint32_t kQsQscale = kQsAlpha + 64 * 4;                   // float[64] query scale * logit scale (log2)
constexpr uint32_t kQsMisc = kQsQscale + 64 * 4;
constexpr uint32_t kQdSmem = kQsMisc + 128;
static_assert(kQdSmem <= 232448, "decode_quant shared memory exceeds the 227 KB per-block limit");
static_assert(kQsRed % 16 == 0 && kQsK % 1024 == 0 && kQsV % 1024 == 0, "alignment");

struct QuantParams {
    const int* seqlens;            // [B]
    const int* page_table;         // [B, max_pages] or null
    const uint16_t* sc;            // [rows][Hkv] pairs of e8m0 bytes (key low, value high)
    const float* gq;               // [512] or null
    const float* gk;
    int* meta;                     // [U][2]
    float* rec_m;
    float* rec_l;
    float* rec_o;
    int B, Hq, Hkv, G, blk, W, Nmax, page_size, max_pages, num_pages, flags, nsplit;
    float scale_log2, eps;
};

// A unit's tiles: nct tiles of 128 entries (cost 1 each), then nwt tiles of 128 raw window tokens (cost
// 2: twice the bytes).
struct QUnit {
    int b, g, nc, nw, nct, nwt, s0;
    __device__ int tiles() const { return nct + nwt; }
    __device__ int cost() const { return nct + 2 * nwt; }
    // first tile that starts at or after cost position x
    __device__ int tile_at(int x) const { return x <= nct ? x : nct + (x - nct + 1) / 2; }
};

__device__ __forceinline__ QUnit q_unit(const QuantParams& p, int u, bool report) {
    QUnit t;
    t.b = u / p.Hkv;
    t.g = u - t.b * p.Hkv;
    int L = __ldg(p.seqlens + t.b);
    if (L < 1) {                                     // 0: a padding row (its merge writes zeros)
        if (report && L < 0) record_error(HCA_ERR_DEVICE_INPUT);
        L = 1;
    }
    const long long a = (long long)L - p.W;          // (t - W + 1) with t = L - 1
    long long nc = a > 0 ? a / p.blk : 0;
    const long long cap = (p.flags & HCA_PAGED) ? (long long)p.max_pages * p.page_size : (long long)p.Nmax;
    if (nc > cap) {
        if (report) record_error(HCA_ERR_DEVICE_INPUT);
        nc = cap;
    }
    t.nc = (int)nc;
    t.nw = L < p.W ? L : p.W;
    t.nct = (t.nc + kDecTile - 1) / kDecTile;
    t.nwt = (t.nw + kDecTile - 1) / kDecTile;
    t.s0 = (p.flags & HCA_WINDOW_RING) ? 0 : p.W - t.nw;
    return t;
}

// Block-wide inclusive scan of one int per thread (all threads of the CTA call it).
__device__ __forceinline__ int q_scan(int v, int* warp_tot, int* total_out) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += n;
    }
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    int pre = 0, tot = 0;
    for (int w = 0; w < kQdThreads / 32; ++w) {
        if (w < warp) pre += warp_tot[w];
        tot += warp_tot[w];
    }
    __syncthreads();
    *total_out = tot;
    return v + pre;
}

// This CTA's tiles in order.  Either one unit's tiles [a, b) (`fixed`), or the tiles that start in the
// cost range [cs, ce) of the batch's list.
struct QIter {
    const QuantParams* p;
    long long ce, pu;              // end of the range; cost position where unit u starts
    QUnit t;
    int u, tb, tend, tile, item, qitem;
    bool fixed, done;

    __device__ void load(long long from) {
        t = q_unit(*p, u, false);
        tb = t.tile_at((int)((from > pu ? from : pu) - pu));
        const long long end = pu + t.cost();
        tend = t.tile_at((int)((ce < end ? ce : end) - pu));
        tile = tb;
    }
    __device__ void init(const QuantParams* pp, int u0, long long p0, long long a, long long b, bool fix) {
        p = pp;
        u = u0;
        pu = p0;
        ce = b;
        fixed = fix;
        item = qitem = 0;
        done = u0 < 0 || a >= b;
        if (done) return;
        if (fixed) {
            t = q_unit(*p, u, false);
            tb = tile = (int)a;
            tend = (int)b;
        } else {
            load(a);
            if (tb >= tend) advance();
        }
    }
    __device__ void advance() {            // to the next unit with a tile in the range
        do {
            pu += t.cost();
            ++u;
            if (fixed || pu >= ce) {
                done = true;
                return;
            }
            load(pu);
        } while (tb >= tend);
    }
    __device__ bool first() const { return tile == tb; }
    __device__ bool last() const { return tile == tend - 1; }
    __device__ bool comp() const { return tile < t.nct; }
    // the query rows are loaded for the first tile of each kind in a piece, and free after its last
    __device__ bool qfirst() const { return tile == tb || tile == t.nct; }
    __device__ bool qlast() const { return tile == tend - 1 || tile == t.nct - 1; }
    __device__ int nvalid() const {
        return comp() ? min(kDecTile, t.nc - tile * kDecTile) : min(kDecTile, t.nw - (tile - t.nct) * kDecTile);
    }
    __device__ void next() {
        if (qlast()) ++qitem;
        if (++tile < tend) return;
        ++item;
        advance();
    }
};

// Page of 64-aligned entry j of a sequence, clamped into the pool (out of it: reported).
__device__ __forceinline__ int q_page(const QuantParams& p, int b, int j, bool report) {
    const int pg = __ldg(p.page_table + (size_t)b * p.max_pages + j / p.page_size);
    if (pg < 0 || pg >= p.num_pages) {
        if (report) record_error(HCA_ERR_DEVICE_INPUT);
        return min(max(pg, 0), p.num_pages - 1);
    }
    return pg;
}

template <bool NORM, bool PAGED>
__global__ void __launch_bounds__(kQdThreads, 1)
decode_quant_kernel(const QuantParams p, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_kw, const __grid_constant__ CUtensorMap tm_vw) {
    extern __shared__ __align__(1024) uint8_t dsmem[];
    // the swizzled operand tiles need a 1024-byte aligned base; there is no room for slack
    if (smem_u32(dsmem) & 1023u) {
        if (threadIdx.x == 0) record_error(HCA_ERR_INTERNAL);
        return;
    }
    uint8_t* sm = dsmem;
    uint64_t* full_k = reinterpret_cast<uint64_t*>(sm + kQsBar);   // [kQdRing] K slab landed
    uint64_t* empty_k = full_k + kQdRing;          // [kQdRing] K slab consumed
    uint64_t* full_v = empty_k + kQdRing;
    uint64_t* empty_v = full_v + kQdRing;
    uint64_t* q_tma = empty_v + kQdRing;           // query rows landed
    uint64_t* q_full = q_tma + 1;                  // query operand ready
    uint64_t* q_empty = q_full + 1;                // query operand no longer read
    uint64_t* s_full = q_empty + 1;                // [kQdLook]
    uint64_t* s_empty = s_full + kQdLook;          // [kQdLook]
    uint64_t* p_full = s_empty + kQdLook;          // [kDecPBufs]
    uint64_t* p_empty = p_full + kDecPBufs;        // [kDecPBufs]
    uint64_t* o_full = p_empty + kDecPBufs;
    uint64_t* o_empty = o_full + 1;
    float* red = reinterpret_cast<float*>(sm + kQsRed);
    float* m_s = reinterpret_cast<float*>(sm + kQsMax);
    float* al_s = reinterpret_cast<float*>(sm + kQsAlpha);
    float* qs_s = reinterpret_cast<float*>(sm + kQsQscale);
    int* misc = reinterpret_cast<int*>(sm + kQsMisc);
    volatile int* abort_flag = misc + 0;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 1);
    int* sched = misc + 2;                         // [0] first unit, [1] aligned, [2 ..] scan scratch

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int U = p.B * p.Hkv;
    const int cta = blockIdx.x;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < kQdRing; ++i) {
            mbar_init(&full_k[i], 1);
            mbar_init(&empty_k[i], 1);
            mbar_init(&full_v[i], 1);
            mbar_init(&empty_v[i], 1);
        }
        mbar_init(q_tma, 1);
        mbar_init(q_full, kDecSoftWarps);
        mbar_init(q_empty, 1);
        for (int i = 0; i < kQdLook; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kDecSoftWarps);
        }
        for (int i = 0; i < kDecPBufs; ++i) {
            mbar_init(&p_full[i], kDecSoftWarps);
            mbar_init(&p_empty[i], 1);
        }
        mbar_init(o_full, 1);
        mbar_init(o_empty, kDecSoftWarps);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    if (threadIdx.x == 32) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_kw);
        prefetch_tmap(&tm_vw);
    }

    // ---- this CTA's tiles.  Two ways to cut the batch, as in decode.cuh:
    //  - unit-aligned, when the batch has no more units than CTAs: unit u gets k_u CTAs, k_u between
    //    1 and its tile count, for the smallest cost per CTA T in tpc .. tpc + 3 whose counts fit the
    //    grid; every CTA then holds one piece (one query load, one record);
    //  - otherwise equal cost ranges of at least 2 (the cost of one window tile), so that every CTA between
    //    a unit's first and last holds one of its tiles and leaves a record.
    const bool small_batch = U <= kQdThreads;
    int my_c = 0, my_t = 0;
    long long total = 0;
    for (int u = threadIdx.x; u < U; u += kQdThreads) {
        const QUnit t = q_unit(p, u, true);
        my_c = t.cost();
        my_t = t.tiles();
        total += my_c;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    {
        long long* wt = reinterpret_cast<long long*>(red);
        if (lane == 0) wt[warp] = total;
        __syncthreads();
        total = 0;
        for (int w = 0; w < kQdThreads / 32; ++w) total += wt[w];
        __syncthreads();
    }
    const long long tpc = max(2ll, (total + p.nsplit - 1) / p.nsplit);
    long long* sched64 = reinterpret_cast<long long*>(red + 64);   // [0] start, [1] end, [2] first unit's position
    unsigned long long* wsum = reinterpret_cast<unsigned long long*>(red);   // [warp]
    int my_k = 0;
    bool aligned = false;
    if (small_batch && U <= p.nsplit && p.nsplit < 0x4000 && total <= 0x3fffffffll) {
        // the four candidate counts are summed in one reduction, as 16-bit fields: k_u <= nsplit *
        // cost_u / total + 2, so each sum is at most nsplit + 2 U < 2^16
        const bool mine = threadIdx.x < U;
        const unsigned fl = mine ? (unsigned)((long long)my_c * p.nsplit / total) : 0u;
        unsigned long long packed = 0;
        if (mine)
#pragma unroll 1
            for (unsigned w = 0; w < 4; ++w) {
                const unsigned T = (unsigned)tpc + w;
                const unsigned k = min((unsigned)my_t, max(fl, ((unsigned)my_c + T - 1u) / T));
                packed |= (unsigned long long)max(1u, k) << (16 * w);
            }
        unsigned long long sum = packed;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) wsum[warp] = sum;
        __syncthreads();
        sum = 0;
        for (int v = 0; v < kQdThreads / 32; ++v) sum += wsum[v];
        __syncthreads();
        for (int w = 3; w >= 0; --w)
            if ((int)((sum >> (16 * w)) & 0xffffu) <= p.nsplit) {
                aligned = true;
                my_k = (int)((packed >> (16 * w)) & 0xffffu);
            }
    }
    if (threadIdx.x == 0) {
        sched[0] = -1;
        sched64[0] = aligned ? 0 : min(total, tpc * cta);
        sched64[1] = aligned ? 0 : min(total, tpc * (cta + 1));
    }
    __syncthreads();
    if (aligned) {
        int tot;
        const int incl = q_scan(my_k, sched + 2, &tot);
        const int cu = incl - my_k;
        if (threadIdx.x < U && cu <= cta && cta < cu + my_k) {
            const QUnit t = q_unit(p, threadIdx.x, false);
            const int i = cta - cu;
            sched[0] = threadIdx.x;
            sched64[2] = 0;
            if (2 * my_k <= my_c) {                // every cost range holds a tile's start
                sched64[0] = t.tile_at((int)((long long)my_c * i / my_k));
                sched64[1] = t.tile_at((int)((long long)my_c * (i + 1) / my_k));
            } else {                               // near one tile per CTA: even tile counts
                sched64[0] = (long long)my_t * i / my_k;
                sched64[1] = (long long)my_t * (i + 1) / my_k;
            }
        }
    } else {
        // the unit holding cost position cs (block-wide scan over units)
        const long long cs = sched64[0];
        long long base = 0;
        for (int c0 = 0; c0 < U; c0 += kQdThreads) {
            const int u = c0 + threadIdx.x;
            const int n = u < U ? q_unit(p, u, false).cost() : 0;
            int tot;
            const int incl = q_scan(n, sched + 2, &tot);
            const long long pu = base + incl - n;
            if (u < U && pu <= cs && cs < pu + n) {
                sched[0] = u;
                sched64[2] = pu;
            }
            base += tot;
        }
    }
    __syncthreads();
    const long long r_beg = sched64[0], r_end = sched64[1], p_first = sched64[2];
    const int u_first = sched[0];
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    constexpr int look = NORM ? kQdLookNorm : kQdLook;
    QIter it;
    it.init(&p, u_first, p_first, r_beg, r_end, aligned);

    if (warp == 0 || warp == 3) {
        // ===================================================== TMA of K (warp 0) or V (warp 3), one thread
        if (lane == 0) {
            const bool is_v = warp == 3;
            uint64_t* full = is_v ? full_v : full_k;
            uint64_t* empty = is_v ? empty_v : empty_k;
            uint8_t* ring = sm + (is_v ? kQsV : kQsK);
            const CUtensorMap* mc = is_v ? &tm_v : &tm_k;
            const CUtensorMap* mw = is_v ? &tm_vw : &tm_kw;
            // test switch (hca_debug_set_drop_slab): the first K slab is never requested
            bool drop = !is_v && *reinterpret_cast<volatile int*>(&g_debug_drop_slab) != 0;
            uint32_t n = 0;
            bool ok = true;
            for (; ok && !it.done; it.next()) {
                const bool comp = it.comp();
                int pg[2] = {0, 0};
                const int j0 = it.tile * kDecTile;
                const bool h1 = j0 + 64 < it.t.nc;
                if (PAGED && comp) {
                    pg[0] = q_page(p, it.t.b, j0, true);
                    pg[1] = h1 ? q_page(p, it.t.b, j0 + 64, true) : pg[0];
                }
                const int ns = comp ? 4 : 8;
                for (int s = 0; s < ns; ++s, ++n) {
                    const uint32_t st = n % kQdRing;
                    if (!mbar_wait(&empty[st], ((n / kQdRing) & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (drop) {          // the slab never lands: its consumer's wait runs out
                        ok = false;
                        break;
                    }
                    uint8_t* dst = ring + st * kSlabBytes;
                    if (PAGED && comp) {
                        mbar_arrive_expect_tx(&full[st], h1 ? 2 * 8192 : 8192);
                        for (int h = 0; h < (h1 ? 2 : 1); ++h)
                            tma_load_4d(dst + h * 8192, mc, &full[st], 128 * s, it.t.g, (j0 + 64 * h) % p.page_size, pg[h]);
                    } else {
                        mbar_arrive_expect_tx(&full[st], kSlabBytes);
                        tma_load_4d(dst, comp ? mc : mw, &full[st], (comp ? 128 : 64) * s, it.t.g,
                                    comp ? j0 : it.t.s0 + (it.tile - it.t.nct) * kDecTile, it.t.b);
                    }
                }
            }
            mbar_drain_ring(full, n, kQdRing);
        }
    } else if (warp == 1) {
        // ===================================================== QK^T issuer (warp waits, lane 0 issues)
        const uint32_t id_w = idesc_bf16(128, kDecHeads, 0, 0), id_wkk = idesc_bf16(128, 128, 0, 0);
        const uint32_t id_e = idesc_f8(128, kDecHeads, kFmtE4M3, kFmtE4M3, 0, 0);
        const uint32_t id_ekk = idesc_f8(128, 128, kFmtE4M3, kFmtE4M3, 0, 0);
        const uint32_t q_base = smem_u32(sm + kQsQ);
        uint32_t ks = 0, nq = 0;
        for (int n = 0; !it.done; it.next(), ++n) {
            const int sb = n % look;
            if (it.qfirst()) {
                // the query rows of the piece (or its window part), once this warp's MMAs no longer read
                // the ones before
                if (!warp_wait(q_empty, (nq & 1) ^ 1, abort_flag)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_tma, kDecQBytes);
                    for (int s = 0; s < kDecSlabs; ++s)
                        tma_load_4d(sm + kQsQ + s * 8192, &tm_q, q_tma, 64 * s, it.t.g * p.G, it.t.b, 0);
                }
                __syncwarp();
                ++nq;
                if (!warp_wait(q_full, it.qitem & 1, abort_flag)) break;
            }
            if (!warp_wait(&s_empty[sb], ((n / look) & 1) ^ 1, abort_flag)) break;
            // the K K^T accumulator has one buffer: wait until tile n-1's softmax has read it
            if (NORM && n > 0 && !warp_wait(&s_empty[(n - 1) % look], ((n - 1) / look) & 1, abort_flag)) break;
            tc_fence_after();
            const uint32_t dst = tmem + dec_s_col(sb);
            const bool comp = it.comp();
            const int ns = comp ? 4 : 8;
            bool ok = true;
            for (int s = 0; s < ns; ++s, ++ks) {
                const uint32_t st = ks % kQdRing;
                if (!warp_wait(&full_k[st], (ks / kQdRing) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t kb = smem_u32(sm + kQsK + st * kSlabBytes);
                    const uint32_t qb = q_base + s * 8192;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t ad = smem_desc_sw128(kb + kk * 32, 16, 1024);
                        const uint64_t bd = smem_desc_sw128(qb + kk * 32, 16, 1024);
                        const uint32_t acc = (s | kk) ? 1u : 0u;
                        if (comp) {
                            mma_f8(dst, ad, bd, id_e, acc);
                            mma_f8(dst, ad, smem_desc_sw128(qb + 32768 + kk * 32, 16, 1024), id_e, 1u);
                            if (NORM) mma_f8(tmem + kTmKK, ad, ad, id_ekk, acc);
                        } else {
                            mma_ss(dst, ad, bd, id_w, acc);
                            if (NORM) mma_ss(tmem + kTmKK, ad, ad, id_wkk, acc);
                        }
                    }
                    mma_commit(&empty_k[st]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (lane == 0) {
                mma_commit(&s_full[sb]);
                if (it.qlast()) mma_commit(q_empty);
            }
            __syncwarp();
        }
        if (lane == 0 && nq) mbar_drain_wait(q_tma, (nq - 1) & 1);
        __syncwarp();
    } else if (warp == 2) {
        // ===================================================== PV issuer (warp waits, lane 0 issues)
        const uint32_t id_w = idesc_bf16(128, kDecHeads, 1, 1);
        const uint32_t id_hi = idesc_f8(128, kDecHeads, kFmtE4M3, kFmtE4M3, 1, 1);
        const uint32_t id_lo = idesc_f8(128, kDecHeads, kFmtE4M3, kFmtE5M2, 1, 1);
        uint32_t vs = 0;
        for (int n = 0; !it.done; it.next(), ++n) {
            const int b = n % kDecPBufs;
            const bool first = it.first(), comp = it.comp();
            if (!warp_wait(&p_full[b], (n / kDecPBufs) & 1, abort_flag)) break;
            if (first && !warp_wait(o_empty, (it.item & 1) ^ 1, abort_flag)) break;
            tc_fence_after();
            const int nvalid = it.nvalid();
            const uint32_t p_base = smem_u32(sm + kQsP + b * kDecPBytes);
            const int per = comp ? 1 : 2;                  // slabs per 128-channel chunk
            bool ok = true;
            for (int c = 0; c < 4; ++c, vs += per) {
                const uint32_t st = vs % kQdRing;          // per == 2: vs is even, the two slabs adjoin
                for (int x = 0; ok && x < per; ++x)
                    ok = warp_wait(&full_v[st + x], (vs / kQdRing) & 1, abort_flag);
                if (!ok) break;
                uint8_t* slab = sm + kQsV + st * kSlabBytes;
                if (nvalid < kDecTile) {
                    // rows >= nvalid may hold anything (memory past the visible entries, ring slots not
                    // yet written): zero them so 0-probability keys contribute exactly 0
                    const int nz = (kDecTile - nvalid) * 8;
                    for (int i = lane; i < per * nz; i += 32) {
                        const int sl = i / nz, k = i - sl * nz;
                        *reinterpret_cast<uint4*>(slab + sl * kSlabBytes + (nvalid + (k >> 3)) * 128 + (k & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t vb = smem_u32(slab);
                    const uint32_t dst = tmem + kTmO + 64 * c;
                    if (comp) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {   // 32 keys each
                            const uint64_t ad = smem_desc_sw128(vb + kk * 4096, kSlabBytes, 1024);
                            mma_f8(dst, ad, smem_desc_sw64(p_base + kk * 2048, 8192, 512), id_hi, (first && kk == 0) ? 0u : 1u);
                            mma_f8(dst, ad, smem_desc_sw64(p_base + 8192 + kk * 2048, 8192, 512), id_lo, 1u);
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)     // 16 keys each
                            mma_ss(dst, smem_desc_sw128(vb + kk * 2048, kSlabBytes, 1024),
                                   smem_desc_sw128(p_base + kk * 2048, 8192, 1024), id_w, (first && kk == 0) ? 0u : 1u);
                    }
                    for (int x = 0; x < per; ++x) mma_commit(&empty_v[st + x]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (lane == 0) {
                mma_commit(&p_empty[b]);
                if (it.last()) mma_commit(o_full);
            }
            __syncwarp();
        }
    } else {
        // ===================================================== softmax / record (8 warps)
        const int q4 = warp & 3;                             // TMEM lane quarter
        const int hh = (warp - kQdSoftWarp0) >> 2;           // head half
        const int h0 = 32 * hh;
        const int r = q4 * 32 + lane;                        // key row within the tile / channel within a chunk
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const int sidx = threadIdx.x - 32 * kQdSoftWarp0;    // 0..255
        // the two scale bytes of this thread's key in the iterator's tile (1.0 for window tokens)
        auto scales = [&]() -> uint32_t {
            if (it.done || !it.comp() || r >= it.nvalid()) return 0x7f7fu;
            const int j = it.tile * kDecTile + r;
            long long row;
            if (PAGED)
                row = (long long)q_page(p, it.t.b, j, false) * p.page_size + j % p.page_size;
            else
                row = (long long)it.t.b * p.Nmax + j;
            return __ldg(p.sc + row * p.Hkv + it.t.g);
        };
        uint32_t sc = scales();
        float lsum[32];       // this thread's share of the row sums, per head
#pragma unroll
        for (int h = 0; h < 32; ++h) lsum[h] = 0.f;
        bool ok = true;
        for (int n = 0; ok && !it.done; ++n) {
            const bool first = it.first(), last = it.last(), comp = it.comp();
            if (it.qfirst()) {
                // ---- the query operand: q (with QK normalisation q / rms(q) * g_q * g_k, since q_hat . k_hat =
                // (q' . k) / rms(k)), as two e4m3 terms for entries, in bf16 for the window.  Four threads per
                // head, 128 channels each, held in registers between the read and the in-place write.
                if (!group_wait(q_tma, it.qitem & 1, abort_flag)) { ok = false; break; }
                const int h = sidx >> 2, part = sidx & 3;
                float inv = 1.f;
                auto chunk = [&](int i) {       // channels 128 part + 8 i .. + 7 of head h
                    return reinterpret_cast<uint4*>(sm + kQsQ + (2 * part + (i >> 3)) * 8192 + sw128(h, i & 7));
                };
                if (NORM) {
                    float ss = 0.f;
#pragma unroll 4
                    for (int i = 0; i < 16; ++i) {
                        const uint4 x = *chunk(i);
                        const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = bf16lo(w4[e]), b2 = bf16hi(w4[e]);
                            ss = fmaf(a, a, fmaf(b2, b2, ss));
                        }
                    }
                    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
                    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
                    inv = rsqrtf(ss * (1.f / kDecD) + p.eps);
                }
                // channels ch, ch + 1 of the query, from the bf16 pair w
                auto value = [&](uint32_t w, int ch) {
                    float2 a = make_float2(bf16lo(w), bf16hi(w));
                    if (NORM) {
                        a.x *= inv * __ldg(p.gq + ch) * __ldg(p.gk + ch);
                        a.y *= inv * __ldg(p.gq + ch + 1) * __ldg(p.gk + ch + 1);
                    }
                    return a;
                };
                if (comp) {
                    float am = 0.f;
#pragma unroll 4
                    for (int i = 0; i < 16; ++i) {
                        const uint4 x = *chunk(i);
                        const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 a = value(w4[e], 128 * part + 8 * i + 2 * e);
                            am = fmaxf(am, fmaxf(q_mag(a.x), q_mag(a.y)));
                        }
                    }
                    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
                    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
                    const uint32_t byte = q_scale_byte(am);
                    const float qi = q_inv_scale(byte);
                    if (part == 0) qs_s[h] = q_scale(byte) * p.scale_log2;
                    // the two terms take the rows' place: all of this thread's codes are made before any row
                    // is overwritten
                    uint32_t hi[32], lo[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint4 x = *chunk(i);
                        const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
                        uint32_t hc[4], lc[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 a = value(w4[e], 128 * part + 8 * i + 2 * e);
                            const float a0 = q_prep(a.x, qi), a1 = q_prep(a.y, qi);
                            hc[e] = cvt_e4m3x2(a0, a1);
                            const float2 f = e4m3x2_f32(hc[e]);
                            lc[e] = cvt_e4m3x2(a0 - f.x, a1 - f.y);
                        }
                        hi[2 * i] = hc[0] | hc[1] << 16;
                        hi[2 * i + 1] = hc[2] | hc[3] << 16;
                        lo[2 * i] = lc[0] | lc[1] << 16;
                        lo[2 * i + 1] = lc[2] | lc[3] << 16;
                    }
                    softmax_bar();           // every row has been read
#pragma unroll
                    for (int i = 0; i < 8; ++i) {        // 16 channels: one 16-byte chunk of hi and of lo
                        uint8_t* dst = sm + kQsQ + part * 8192 + sw128(h, i);
                        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                        *reinterpret_cast<uint4*>(dst + 32768) =
                            make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                    }
                    fence_proxy_async_smem();
                    // a unit's entries come first in its piece: the sums start here
#pragma unroll
                    for (int hx = 0; hx < 32; ++hx) lsum[hx] = 0.f;
                } else if (NORM) {
                    if (part == 0) qs_s[h] = p.scale_log2;
#pragma unroll 4
                    for (int i = 0; i < 16; ++i) {
                        uint4* ptr = chunk(i);
                        const uint4 x = *ptr;
                        uint32_t w4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 a = value(w4[e], 128 * part + 8 * i + 2 * e);
                            w4[e] = pack_bf16x2(a.x, a.y);
                        }
                        *ptr = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                    }
                    fence_proxy_async_smem();
                } else if (sidx < 64) {
                    qs_s[sidx] = p.scale_log2;
                }
                softmax_bar();               // qs_s
                if (lane == 0) mbar_arrive(q_full);
            }

            const int sb = n % look;
            const bool valid = r < it.nvalid();
            if (!group_wait(&s_full[sb], (n / look) & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            float z[32];
            tmem_ld16(tmem + lane_off + dec_s_col(sb) + h0, z);
            tmem_ld16(tmem + lane_off + dec_s_col(sb) + h0 + 16, z + 16);
            float kscale = q_scale(sc & 0xffu);
            if (NORM) {
                float d[32];
                tmem_ld16(tmem + lane_off + kTmKK + q4 * 32, d);
                tmem_ld16(tmem + lane_off + kTmKK + q4 * 32 + 16, d + 16);
                tmem_wait_ld();
                float diag = 0.f;
#pragma unroll
                for (int j = 0; j < 32; ++j) diag = (j == lane) ? d[j] : diag;
                kscale *= rsqrtf(diag * (1.f / kDecD) * kscale * kscale + p.eps);
            } else {
                tmem_wait_ld();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[sb]);
            // y = logit + log2(vscale)
            const float lv = (float)((int)(sc >> 8) - 127);
            const float rv = q_inv_scale(sc >> 8);
#pragma unroll
            for (int h = 0; h < 32; h += 4) {
                const float4 qs = *reinterpret_cast<const float4*>(qs_s + h0 + h);
                z[h] = valid ? fmaf(z[h] * kscale, qs.x, lv) : -INFINITY;
                z[h + 1] = valid ? fmaf(z[h + 1] * kscale, qs.y, lv) : -INFINITY;
                z[h + 2] = valid ? fmaf(z[h + 2] * kscale, qs.z, lv) : -INFINITY;
                z[h + 3] = valid ? fmaf(z[h + 3] * kscale, qs.w, lv) : -INFINITY;
            }

            // ---- reference m (shared m_s[64]): the first tile's maximum, then only when some y
            // exceeds it by 2^8
            bool need;
            if (first) {
                need = true;
            } else {
                bool mine = false;
#pragma unroll
                for (int h = 0; h < 32; h += 4) {
                    const float4 mm = *reinterpret_cast<const float4*>(m_s + h0 + h);
                    mine |= (z[h] > mm.x + kRescaleThreshold) | (z[h + 1] > mm.y + kRescaleThreshold) |
                            (z[h + 2] > mm.z + kRescaleThreshold) | (z[h + 3] > mm.w + kRescaleThreshold);
                }
                need = softmax_any(mine);
            }
            if (need) {
                const float tmax = colreduce32<true>(z, lane);
                red[q4 * 64 + h0 + lane] = tmax;
                softmax_bar();
                if (sidx < 64) {
                    const float mo = first ? -INFINITY : m_s[sidx];
                    const float mt = fmaxf(fmaxf(red[sidx], red[64 + sidx]), fmaxf(red[128 + sidx], red[192 + sidx]));
                    const float mn = fmaxf(mo, mt - kQdShift);
                    al_s[sidx] = first ? 0.f : ex2(mo - mn);
                    m_s[sidx] = mn;
                }
                softmax_bar();
                if (!first) {
#pragma unroll
                    for (int h = 0; h < 32; ++h) lsum[h] *= al_s[h0 + h];
                    // rescale O^T once the previous PV has landed
                    const int pb = (n - 1) % kDecPBufs;
                    if (!group_wait(&p_empty[pb], ((n - 1) / kDecPBufs) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
#pragma unroll 1
                        for (int c16 = 0; c16 < 32; c16 += 16) {
                            float o[16];
                            const uint32_t ta = tmem + lane_off + kTmO + 64 * c + h0 + c16;
                            tmem_ld16(ta, o);
                            tmem_wait_ld();
                            uint32_t w[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(o[j] * al_s[h0 + c16 + j]);
                            tmem_st16(ta, w);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
            }
            // ---- probabilities (times vscale) and this thread's row sums
#pragma unroll
            for (int h = 0; h < 32; h += 4) {
                const float4 mm = *reinterpret_cast<const float4*>(m_s + h0 + h);
                z[h] = ex2(z[h] - mm.x);
                z[h + 1] = ex2(z[h + 1] - mm.y);
                z[h + 2] = ex2(z[h + 2] - mm.z);
                z[h + 3] = ex2(z[h + 3] - mm.w);
#pragma unroll
                for (int e = 0; e < 4; ++e) lsum[h + e] = fmaf(z[h + e], rv, lsum[h + e]);
            }
            const int pbuf = n % kDecPBufs;
            if (!group_wait(&p_empty[pbuf], ((n / kDecPBufs) & 1) ^ 1, abort_flag)) { ok = false; break; }
            uint8_t* pt = sm + kQsP + pbuf * kDecPBytes;
            if (comp) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float* y = z + 16 * c + 4 * e;
                        const uint32_t c0 = cvt_e4m3x2(y[0], y[1]), c1 = cvt_e4m3x2(y[2], y[3]);
                        const float2 f0 = e4m3x2_f32(c0), f1 = e4m3x2_f32(c1);
                        hi[e] = c0 | c1 << 16;
                        lo[e] = cvt_e5m2x2(y[0] - f0.x, y[1] - f0.y) | cvt_e5m2x2(y[2] - f1.x, y[3] - f1.y) << 16;
                    }
                    *reinterpret_cast<uint4*>(pt + sw64(r, 2 * hh + c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(pt + 8192 + sw64(r, 2 * hh + c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4*>(pt + sw128(r, 4 * hh + c)) =
                        make_uint4(pack_bf16x2(z[8 * c], z[8 * c + 1]), pack_bf16x2(z[8 * c + 2], z[8 * c + 3]),
                                   pack_bf16x2(z[8 * c + 4], z[8 * c + 5]), pack_bf16x2(z[8 * c + 6], z[8 * c + 7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[pbuf]);

            if (last) {
                // ---- end of this CTA's piece of unit u: the row sums over all key rows, then the
                // record (reference, sum, unnormalised O^T)
                const int u = it.u;
                const int rec = cta + u;
                const float tsum = colreduce32<false>(lsum, lane);
                red[q4 * 64 + h0 + lane] = tsum;
                softmax_bar();
                if (sidx == 0) {
                    if (it.tb == 0) p.meta[2 * u] = cta;
                    if (it.tend == it.t.tiles()) p.meta[2 * u + 1] = cta;
                }
                if (sidx < 64) {
                    p.rec_m[(size_t)rec * 64 + sidx] = m_s[sidx];
                    p.rec_l[(size_t)rec * 64 + sidx] = (red[sidx] + red[64 + sidx]) + (red[128 + sidx] + red[192 + sidx]);
                }
                softmax_bar();     // red[] is free again before the next piece's first reduction
#pragma unroll
                for (int h = 0; h < 32; ++h) lsum[h] = 0.f;
                if (!group_wait(o_full, it.item & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                float* orec = p.rec_o + (size_t)rec * 64 * kDecD;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
#pragma unroll 1
                    for (int c16 = 0; c16 < 32; c16 += 16) {
                        float o[16];
                        tmem_ld16(tmem + lane_off + kTmO + 64 * c + h0 + c16, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int h = h0 + c16 + j;
                            if (h < p.G) orec[(size_t)h * kDecD + 128 * c + r] = o[j];
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_empty);
            }
            it.next();
            sc = scales();
        }
    }

    __syncwarp();      // every role reconverges its warp before the CTA-wide barrier
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace hca
