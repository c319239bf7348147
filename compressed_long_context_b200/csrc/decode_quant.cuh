// decode_quant.cuh -- split-KV HCA decode over an 8-bit compressed cache (hca_decode_quant).
//
// Same operation and work decomposition as decode.cuh (one query per sequence over its entries and its
// raw window, the batch's key tiles cut into one range per CTA, partial records merged afterwards); the
// entries are e4m3 codes with one power-of-two scale per key and per value vector (fp8.cuh), the window
// is raw bf16.  Entries go from memory to the tensor cores as they are (kind::f8f6f4, K = 32): widening
// them on the way would cost more shared-memory bandwidth than HBM delivers bytes (write 64 KB, read 64 KB,
// write 128 KB, read 128 KB per 128 keys of K and again of V).  The other operands are bf16 quantities, so
// each is split into two 8-bit terms, both multiplied with the same 8-bit tile in fp32:
//   q = hi + lo, both e4m3, after a power-of-two scale per head that puts max|q| in (224, 448].  hi keeps 4
//       significant bits and lo the next 4: a bf16 query (8 bits) is represented exactly down to 2^-10 of its
//       head's largest channel, and to 2^-18.8 of that channel below.  Same rounding (2^-8 at most) as bf16
//       for the fp32 queries that QK normalisation makes.
//   p = hi (e4m3) + lo (e5m2): where hi is normal (p >= 2^-6, 2^-10 of the row's largest) at most 2^-4 * 2^-3 =
//       2^-7 off, 2^-10 in the mean square; below, hi is within 2^-10 and lo within 2^-3 of the rest: 2^-13, or
//       2^-17 of the largest.  lo is e5m2 because its range matters more than its last bit: a probability down to
//       2^-20 of the largest still has a term, so a long tail of small probabilities is kept.
//   (bf16 keys: p as two bf16 terms, 2^-16, in the two P buffers: one term would be 2^-8 off, as much as the output's own
//   rounding; short sequences, whose window weighs most, were 1.7 times further off with QK normalisation.)
// The scale of a value vector belongs to the key, which is the contraction's axis, so it goes into p: with
// y = z + log2(vscale), the accumulators hold sums of 2^(y - m) * code, the reference m is the running
// maximum of y, and the row sum l adds 2^(y - m) / vscale = 2^(z - m).  m is kept 2^4 below the maximum
// and moves when some y exceeds it by 2^8, so that p <= 256 and 2^4 for the largest key: e4m3 ends at 448.  (2^6
// moved it, and with it 128 KB of accumulators, in most tiles of the ragged batch: 4 % of its time.)
// The same kernel with bf16 entries (E8 = false) attends what the sequences of hca_decode_shared do not have in
// common: then all tiles are of the window's kind, and the reference moves at 2^32 (bf16 holds any p).
//
// Inside a CTA (12 warps: a thirteenth would leave 128 registers per thread instead of 168):
//   warp 0, 3   TMA of K / of V: slabs of 16 KB (128 keys x 128 codes, or x 64 bf16 channels) through a ring of
//               four each; a tile of codes fills a ring once, a bf16 tile twice;
//   warp 1      TMA of the query rows, once per (unit, kind of tile): 8-bit hi / lo for codes (made in place by
//               the softmax warps), bf16 otherwise;  tcgen05.mma  S^T[128 keys x 64 heads] = K Q^T;
//   warp 2      the CTA's range of tiles, then tcgen05.mma  O^T[512 x 64] += V^T P^T over the 32-key (bf16: 16-key)
//               steps that hold a key;
//   warps 4-11  softmax, two per TMEM lane quarter, thread = (key row, 32 heads); record at a piece's end.
//
// What bounds it.  A small call: its chain of first steps, whose code is fetched cold (about 30 cycles an instruction).
// So they are loops, not unrolled, the range is found by one warp, and the MMA issuers are elected: one 4K sequence
// (one tile of each kind on two CTAs) takes 17.3 us with the merge, where unrolled set-up code and issuers chosen by
// lane took 27.  A large one: 3.0 us for each tile of codes from memory (6.5 TB/s while all SMs stream; 2.9 from L2, with QK
// normalisation 3.7 and 3.3; the MMAs take 1.6 to 1.9, bound by the shared memory that they read: an M = 128, N = 64 MMA
// takes 48 cycles), and 8 us at each start of a unit, which nothing hides.  256 sequences of 128K: 84 us and the merge, 4.7 TB/s
// of memory over it all, every code read once, tensor pipe 24 % active.  Requesting tiles into L2 ahead of the rings changed
// nothing at 1, 2 or 3 tiles.
#pragma once

#include "decode.cuh"
#include "fp8.cuh"
#include "merge.cuh"

namespace hca {

constexpr int kQdThreads = 384;
constexpr int kQdSoftWarp0 = 4;
constexpr int kQdRing = 4;                 // slabs per ring (K, V)
constexpr int kQdLook = 4;                 // S buffers at most
// Tensor memory: S buffers (and K K^T) in columns 0 .. 255, O^T in 256 .. 511 (4 x 64 for 128 channels each).
constexpr uint32_t kQdKK = 128, kQdO = 256;
constexpr int kQdKept = 2048;              // units whose tile counts fit the P buffers while these are not in use
// Cost of starting a unit, in tiles: query operand, refilled pipeline and record take about 8 us, a tile 3.  It lies before
// the unit's first tile, so a range that starts units holds fewer tiles.  128 sequences of 4K to 1M tokens with QK
// normalisation, 256 and 160 of 128K: 159, 108 and 75.6 us; with a start of one tile 158, 110 and 75.3, of three 155, 108 and 79.
constexpr int kQdStart = 2;
constexpr float kQdShift = 4.0f;           // the reference m lies this far (log2) below the maximum

// Shared memory: query operand (8 tiles of 8 KB: 64 bf16 channels of each head, or 128 codes) and K ring, 64 KB each; P
// buffers; V ring.
constexpr uint32_t kQdQTile = 8192;
constexpr uint32_t kQsQ = 0;
constexpr uint32_t kQsP = kDecQBytes + kQdRing * kSlabBytes;
constexpr uint32_t kQsV = kQsP + kDecPBufs * kDecPBytes;
constexpr uint32_t kQsBar = kQsV + kQdRing * kSlabBytes;
constexpr int kQdBars = 4 * kQdRing + 3 + 2 * kQdLook + 2 * kDecPBufs + 2;
constexpr uint32_t kQsRed = (kQsBar + kQdBars * 8 + 127) & ~127u;   // float[4][64]
constexpr uint32_t kQsMax = kQsRed + 4 * 64 * 4;                    // float[64] reference m per head
constexpr uint32_t kQsAlpha = kQsMax + 64 * 4;                      // float[64] rescale factors
constexpr uint32_t kQsQscale = kQsAlpha + 64 * 4;                   // float[64] query scale * logit scale (log2)
constexpr uint32_t kQsMisc = kQsQscale + 64 * 4;
constexpr uint32_t kQdSmem = kQsMisc + 128;
static_assert(kQdKept * 8 <= kDecPBufs * kDecPBytes, "kept tile counts fit the P buffers");
static_assert(kQdSmem <= 232448, "decode_quant shared memory exceeds the 227 KB per-block limit");
static_assert(kQsRed % 16 == 0 && kQsP % 1024 == 0 && kQsV % 1024 == 0, "alignment");

// Codes with QK normalisation ("joined"): two tiles of the query operand and a slot of the K ring alternate, so that slab s of
// a tile of codes, which always lies in slot s, continues q hi and q lo of its channels: one MMA of N = 256 multiplies the slab
// with hi, lo and itself, into one buffer of [hi 64 | lo 64 | K K^T 128] columns.  It takes 128 cycles, where three MMAs take
// 48 + 48 + 64 (128 ragged sequences 164.7 -> 161.1 us).  Else the operand lies in front of the ring, hi and lo go into one
// accumulator, and the S buffers have 64 columns: the alternating layout was slower there, with one MMA of N = 128 or two of
// N = 64 (64 sequences of 128K 40.0 against 39.4 us).
template <bool NORM, bool E8>
struct QdShape {
    static constexpr bool kJoined = NORM && E8;
    static constexpr int kLook = kJoined ? 1 : (NORM ? 2 : 4);                                // S buffers
    static constexpr uint32_t kK = kJoined ? 2 * kQdQTile : kDecQBytes;                       // K slot s at kK + s * kSlot
    static constexpr uint32_t kSlot = kJoined ? 2 * kQdQTile + kSlabBytes : kSlabBytes;
    static constexpr uint32_t kHi = kJoined ? kSlot : kQdQTile;                               // q hi of slab s at s * kHi
    static constexpr uint32_t kLo = kJoined ? kQdQTile : 4 * kQdQTile;                        // q lo behind q hi
    // tile s of the bf16 operand
    __host__ __device__ static constexpr uint32_t q_tile(uint32_t s) {
        return kJoined ? (s >> 1) * kSlot + (s & 1) * kQdQTile : s * kQdQTile;
    }
};
static_assert(2 * kQdQTile == kSlabBytes && 8 * kQdQTile == kDecQBytes, "operand tiles and slots share one aligned grid");

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
    int cap;                       // entries that a sequence's cache can hold
    int skip;                      // the cache holds the entries from this one on (0: all)
    // hca_decode_shared: this pass runs beside the prefix pass on the SMs that it leaves (0: alone on all)
    long long pfx_total;
    int pfx_max;
    SharedPlan* plan;              // written for the merge
    float scale_log2, eps;
};

// Keys of a sequence of length L: nc own entries visible (clamped into the cache), nw window tokens.
struct QKeys {
    int nc, nw;
};

// Not inlined: a dozen callers share its code, which the first of them fetches.
__device__ __noinline__ QKeys q_keys_of(int L, int W, int blk, int skip, int cap, bool report) {
    if (L < 1) {                                     // 0: a padding row (its merge writes zeros)
        if (report && L < 0) record_error(HCA_ERR_DEVICE_INPUT);
        L = 1;
    }
    const int a = L - W;                           // (t - W + 1) with t = L - 1
    int nc = (a > 0 ? (int)((unsigned)a / (unsigned)blk) : 0) - skip;
    nc = nc > 0 ? nc : 0;
    if (nc > cap) {
        if (report) record_error(HCA_ERR_DEVICE_INPUT);
        nc = cap;
    }
    return QKeys{nc, L < W ? L : W};
}
__device__ __forceinline__ QKeys q_keys(const QuantParams& p, int L, bool report) {
    return q_keys_of(L, p.W, p.blk, p.skip, p.cap, report);
}

__device__ __forceinline__ float q_warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// A unit's tiles: nct tiles of 128 entries (cost 1 each), then nwt tiles of 128 raw window tokens (cost
// WC: 2 beside codes, which have half the bytes, else 1).  All counts of a batch fit 31 bits (checked on the host).
struct QTiles {
    int nct, nwt;
    __device__ __forceinline__ int tiles() const { return nct + nwt; }
    template <int WC> __device__ __forceinline__ int cost() const { return nct + WC * nwt; }
    // first tile that starts at or after cost position x (from the first tile on)
    template <int WC> __device__ __forceinline__ int tile_at(int x) const {
        return x <= nct ? max(x, 0) : nct + (x - nct + WC - 1) / WC;
    }
};
__device__ __forceinline__ QTiles q_tiles(const QKeys& k) {
    return QTiles{(k.nc + kDecTile - 1) / kDecTile, (k.nw + kDecTile - 1) / kDecTile};
}
__device__ __forceinline__ int q_seq(const QuantParams& p, int u) { return p.Hkv == 1 ? u : u / p.Hkv; }

// A CTA's range: either tiles [beg, end) of unit u (`aligned`), or the tiles that start in the cost range [beg, end) of
// the batch's list, in which unit u starts at pu.
struct QRange {
    int beg, end, pu, u, aligned;
};

// x * i / k without leaving 32 bits (i <= k < 2^15)
__device__ __forceinline__ int q_part(int x, int i, int k) { return x / k * i + x % k * i / k; }

__device__ __forceinline__ int q_scan(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += n;
    }
    return v;
}

// Found by one warp.  Two ways to cut the batch, as in decode.cuh:
//  - unit-aligned, when the batch has no more units than CTAs: unit u gets k_u CTAs, k_u between 1 and its tile count,
//    for the smallest cost per CTA T in tpc .. tpc + 3 whose counts fit the grid; every CTA then holds one piece
//    (one query load, one record);
//  - otherwise equal cost ranges of at least the cost of a window tile, so that every CTA between a unit's first
//    tile and its last holds one of its tiles and leaves a record.
template <int WC>
__device__ __forceinline__ void q_range(const QuantParams& p, int cta, int grid, QRange* out, uint2* kept) {
    const int lane = threadIdx.x & 31;
    const int U = p.B * p.Hkv;
    // the first kQdKept units' tile counts are kept in shared memory for the passes below
    int total = 0;
#pragma unroll 1
    for (int u0 = lane; u0 < U; u0 += 128) {
        int L[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) L[i] = u0 + 32 * i < U ? __ldg(p.seqlens + q_seq(p, u0 + 32 * i)) : 1;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const int u = u0 + 32 * i;
            if (u >= U) break;
            const QTiles t = q_tiles(q_keys(p, i == 0 ? L[0] : i == 1 ? L[1] : i == 2 ? L[2] : L[3], true));
            total += t.cost<WC>();
            if (u < kQdKept) kept[u] = make_uint2(t.nct, t.nwt);
        }
    }
    total = __reduce_add_sync(0xffffffffu, total);
    __syncwarp();
    auto tiles_of = [&](int u) {
        if (u < kQdKept) {
            const uint2 t = kept[u];
            return QTiles{(int)t.x, (int)t.y};
        }
        return q_tiles(q_keys(p, __ldg(p.seqlens + q_seq(p, u)), false));
    };
    int nsplit = p.nsplit;
    if (p.pfx_total > 0) {
        const SharedPlan plan = shared_plan_warp(p.pfx_total, total, U, p.pfx_max, p.nsplit);
        nsplit = min(plan.splits, grid);
        if (lane == 0 && cta == 0) *p.plan = plan;
    }
    int tpc = (int)(((unsigned)total + nsplit - 1u) / (unsigned)nsplit);
    int w = 4;
    const float share = (float)nsplit / (float)total;
    auto count = [&](const QTiles& t, int x) {
        const int c = t.cost<WC>();
        return max(1, min(t.tiles(), max((int)((float)c * share), (int)(((unsigned)c + (unsigned)(tpc + x) - 1u) / (unsigned)(tpc + x)))));
    };
    if (U <= nsplit && nsplit < 0x2000) {
        // two candidate counts to a word: k_u <= nsplit * cost_u / total + 2 (one more for the rounding of `share`), so
        // each sum is at most nsplit + 3 U < 2^15
#pragma unroll 1
        for (int x = 0; x < 4 && w == 4; x += 2) {
            unsigned sum = 0;
#pragma unroll 1
            for (int u = lane; u < U; u += 32) {
                const QTiles t = tiles_of(u);
                sum += (unsigned)count(t, x) | (unsigned)count(t, x + 1) << 16;
            }
            sum = __reduce_add_sync(0xffffffffu, sum);
            w = (int)(sum & 0xffffu) <= nsplit ? x : (int)(sum >> 16) <= nsplit ? x + 1 : 4;
        }
    }
    // the unit that holds this CTA (aligned: in the list of counts) or cost position beg
    QRange r = {0, 0, 0, -1, 0};
    if (w == 4) {
        total += kQdStart * U;
        tpc = max(WC, (int)(((unsigned)total + nsplit - 1u) / (unsigned)nsplit));
        r.beg = (int)min((long long)total, (long long)tpc * cta);
        r.end = (int)min((long long)total, (long long)tpc * (cta + 1));
    }
    const int at = w < 4 ? cta : r.beg;
    int base = 0;
    bool found = w == 4 && r.beg >= r.end;
#pragma unroll 1
    for (int u0 = 0; u0 < U && !found; u0 += 32) {
        const int u = u0 + lane;
        QTiles t = {};
        int n = 0;
        if (u < U) {
            t = tiles_of(u);
            n = w < 4 ? count(t, w) : kQdStart + t.cost<WC>();
        }
        const int incl = q_scan(n);
        const int i = at - (base + incl - n);
        const bool mine = i >= 0 && i < n;
        if (mine) {
            r.u = u;
            r.pu = base + incl - n;
            if (w < 4) {
                const int c = t.cost<WC>(), m = t.tiles();
                const bool even = WC * n > c;           // near one tile per CTA: even tile counts, else every cost
                r.beg = even ? q_part(m, i, n) : t.tile_at<WC>(q_part(c, i, n));           // range holds a tile's start
                r.end = even ? q_part(m, i + 1, n) : t.tile_at<WC>(q_part(c, i + 1, n));
                r.aligned = 1;
            }
            *out = r;
        }
        found = __any_sync(0xffffffffu, mine);
        if (found) return;
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) *out = r;                            // nothing to do (u = -1)
}

// This CTA's tiles in order.
template <bool E8>
struct QIter {
    static constexpr int WC = E8 ? 2 : 1;
    const QuantParams* p;
    int ce, pu;                    // end of the range; cost position where unit u starts
    struct {
        int b, g, nc, nw, nct, s0;
    } t;
    int u, tb, tend, ntiles, tile, item;
    bool fixed, done;

    __device__ __forceinline__ void load(int from, const QRange* r) {
        t.b = q_seq(*p, u);
        t.g = u - t.b * p->Hkv;
        const QKeys k = q_keys(*p, __ldg(p->seqlens + t.b), false);
        const QTiles n = q_tiles(k);
        t.nc = k.nc;
        t.nw = k.nw;
        t.nct = n.nct;
        t.s0 = (p->flags & HCA_WINDOW_RING) ? 0 : p->W - k.nw;
        ntiles = n.tiles();
        const int cost = kQdStart + n.template cost<WC>();
        if (fixed && r) {
            tb = r->beg;
            tend = r->end;
        } else {
            tb = n.template tile_at<WC>(from - pu - kQdStart);
            tend = n.template tile_at<WC>(min(ce - pu, cost) - kQdStart);
        }
        tile = tb;
        next_pu = pu + cost;
    }
    int next_pu;
    __device__ __forceinline__ void init(const QuantParams* pp, const QRange& r) {
        p = pp;
        u = r.u;
        pu = r.pu;
        ce = r.end;
        fixed = r.aligned;
        item = 0;
        done = r.u < 0 || r.beg >= r.end;
        if (done) return;
        load(r.beg, &r);
        if (tb >= tend) advance();
    }
    __device__ __forceinline__ void advance() {         // to the next unit with a tile in the range
        do {
            pu = next_pu;
            ++u;
            if (fixed || pu >= ce) {
                done = true;
                return;
            }
            load(pu, nullptr);
        } while (tb >= tend);
    }
    __device__ bool first() const { return tile == tb; }
    __device__ bool last() const { return tile == tend - 1; }
    __device__ bool comp() const { return tile < t.nct; }
    __device__ bool codes() const { return E8 && tile < t.nct; }
    // the query rows are loaded for the first tile of each kind in a piece, and free after its last
    __device__ bool qfirst() const { return tile == tb || (E8 && tile == t.nct); }
    __device__ bool qlast() const { return tile == tend - 1 || (E8 && tile == t.nct - 1); }
    __device__ int nvalid() const {
        return comp() ? min(kDecTile, t.nc - tile * kDecTile) : min(kDecTile, t.nw - (tile - t.nct) * kDecTile);
    }
    __device__ void next() {
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

template <bool NORM, bool PAGED, bool E8>
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
    uint64_t* q_full = q_tma + 1;                  // query operand made from them
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
    QRange* range = reinterpret_cast<QRange*>(misc + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    // bf16 probabilities hold any range: the reference starts at the maximum and moves late
    constexpr float shift = E8 ? kQdShift : 0.f, thr = E8 ? kRescaleThreshold : 32.f;

    if (warp == 2) {
        q_range<E8 ? 2 : 1>(p, cta, gridDim.x, range, reinterpret_cast<uint2*>(sm + kQsP));
    } else if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
    } else if (warp == 0) {
        if (lane == 0) *abort_flag = 0;
        // barriers in order: full / empty of K, of V; q_tma, q_full, q_empty; s_full; s_empty; p_full; p_empty; o_full, o_empty
        for (int i = lane; i < kQdBars; i += 32) {
            const int j = i - 4 * kQdRing;
            const bool many = j == 1 || (j >= 3 + kQdLook && j < 3 + 2 * kQdLook + kDecPBufs) || i == kQdBars - 1;
            mbar_init(&full_k[i], many ? kDecSoftWarps : 1);
        }
        fence_mbar_init();
    } else if (threadIdx.x == 96) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_kw);
        prefetch_tmap(&tm_vw);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    using Shape = QdShape<NORM, E8>;
    constexpr int look = Shape::kLook;
    constexpr bool joined = Shape::kJoined;
    QIter<E8> it;
    it.init(&p, *range);

    if (warp == 0 || warp == 3) {
        // ===================================================== TMA of K (warp 0) or V (warp 3), one thread
        if (elect_one()) {
            const bool is_v = warp == 3;
            uint64_t* full = is_v ? full_v : full_k;
            uint64_t* empty = is_v ? empty_v : empty_k;
            uint8_t* ring = sm + (is_v ? kQsV : Shape::kK);
            const uint32_t slot = is_v ? kSlabBytes : Shape::kSlot;
            const CUtensorMap* mc = is_v ? &tm_v : &tm_k;
            const CUtensorMap* mw = is_v ? &tm_vw : &tm_kw;
            // test switch (hca_debug_set_drop_slab): the first K slab is never requested
            const bool drop = !is_v && *reinterpret_cast<volatile int*>(&g_debug_drop_slab) != 0;
            uint32_t n = 0;
            bool ok = true;
            for (; ok && !it.done; it.next()) {
                const bool comp = it.comp(), halves = PAGED && comp;
                int pg[2] = {0, 0};
                const int j0 = it.tile * kDecTile;
                const bool h1 = j0 + 64 < it.t.nc;
                if (halves) {
                    pg[0] = q_page(p, it.t.b, j0, true);
                    pg[1] = h1 ? q_page(p, it.t.b, j0 + 64, true) : pg[0];
                }
                const int ns = it.codes() ? 4 : 8, wide = it.codes() ? 128 : 64;
                const int row = comp ? j0 : it.t.s0 + (it.tile - it.t.nct) * kDecTile;
#pragma unroll 1
                for (int s = 0; s < ns; ++s, ++n) {
                    const uint32_t st = n % kQdRing;
                    if (!mbar_wait(&empty[st], ((n / kQdRing) & 1) ^ 1, abort_flag) || drop) {   // dropped: its
                        ok = false;                                                  // consumer's wait runs out
                        break;
                    }
                    uint8_t* dst = ring + st * slot;
                    mbar_arrive_expect_tx(&full[st], halves && !h1 ? kSlabBytes / 2 : kSlabBytes);
                    if (halves) {
                        tma_load_4d(dst, mc, &full[st], wide * s, it.t.g, j0 % p.page_size, pg[0]);
                        if (h1) tma_load_4d(dst + 8192, mc, &full[st], wide * s, it.t.g, (j0 + 64) % p.page_size, pg[1]);
                    } else {
                        tma_load_4d(dst, comp ? mc : mw, &full[st], wide * s, it.t.g, row, it.t.b);
                    }
                }
            }
            mbar_drain_ring(full, n, kQdRing);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ===================================================== QK^T issuer (warp waits, one lane issues)
        const uint32_t id_w = idesc_bf16(128, kDecHeads, 0, 0), id_wkk = idesc_bf16(128, 128, 0, 0);
        const uint32_t id_e = idesc_f8(128, joined ? 256 : kDecHeads, kFmtE4M3, kFmtE4M3, 0, 0);
        const uint32_t q_base = smem_u32(sm + kQsQ);
        uint32_t ks = 0, nq = 0, nconv = 0;
        for (int n = 0; !it.done; it.next(), ++n) {
            const int sb = n % look;
            const bool codes = it.codes();
            if (it.qfirst()) {
                // the query rows of the piece (or its window part), once this warp's MMAs no longer read
                // the ones before
                if (!warp_wait(q_empty, (nq & 1) ^ 1, abort_flag)) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(q_tma, kDecQBytes);
#pragma unroll 1
                    for (int s = 0; s < kDecSlabs; ++s)
                        tma_load_4d(sm + kQsQ + Shape::q_tile(s), &tm_q, q_tma, 64 * s, it.t.g * p.G, it.t.b, 0);
                }
                __syncwarp();
                ++nq;
                if (NORM || codes) {
                    if (!warp_wait(q_full, nconv & 1, abort_flag)) break;
                    ++nconv;
                } else if (!warp_wait(q_tma, (nq - 1) & 1, abort_flag)) {
                    break;
                }
            }
            if (!warp_wait(&s_empty[sb], ((n / look) & 1) ^ 1, abort_flag)) break;
            // the K K^T accumulator has one buffer: wait until tile n-1's softmax has read it
            if (NORM && n > 0 && !warp_wait(&s_empty[(n - 1) % look], ((n - 1) / look) & 1, abort_flag)) break;
            tc_fence_after();
            const uint32_t dst = tmem + 64 * sb;
            const int ns = codes ? 4 : 8;
            bool ok = true;
#pragma unroll 1
            for (int s = 0; s < ns; ++s, ++ks) {
                const uint32_t st = ks % kQdRing;
                if (!warp_wait(&full_k[st], (ks / kQdRing) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t kd = smem_desc_sw128(smem_u32(sm + Shape::kK + st * Shape::kSlot), 16, 1024);
                const uint32_t q_off = codes ? s * Shape::kHi : Shape::q_tile(s);
                const uint64_t qd = smem_desc_sw128(q_base + q_off, 16, 1024);
                if (elect_one()) {
                    // descriptors advance by 32 bytes (2 of their units) per step
                    if (E8 && codes) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            mma_f8(dst, kd + 2 * kk, qd + 2 * kk, id_e, (s | kk) ? 1u : 0u);
                            if (!joined) mma_f8(dst, kd + 2 * kk, qd + (Shape::kLo >> 4) + 2 * kk, id_e, 1u);
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            mma_ss(dst, kd + 2 * kk, qd + 2 * kk, id_w, (s | kk) ? 1u : 0u);
                            if (NORM) mma_ss(tmem + kQdKK, kd + 2 * kk, kd + 2 * kk, id_wkk, (s | kk) ? 1u : 0u);
                        }
                    }
                    mma_commit(&empty_k[st]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) {
                mma_commit(&s_full[sb]);
                if (it.qlast()) mma_commit(q_empty);
            }
            __syncwarp();
        }
        if (lane == 0 && nq) mbar_drain_wait(q_tma, (nq - 1) & 1);
        __syncwarp();
    } else if (warp == 2) {
        // ===================================================== PV issuer (warp waits, one lane issues)
        const uint32_t id_w = idesc_bf16(128, kDecHeads, 1, 1);
        const uint32_t id_hi = idesc_f8(128, kDecHeads, kFmtE4M3, kFmtE4M3, 1, 1);
        const uint32_t id_lo = idesc_f8(128, kDecHeads, kFmtE4M3, kFmtE5M2, 1, 1);
        uint32_t vs = 0, pn = 0;                           // V slabs, P buffers used
        for (; !it.done; it.next()) {
            const bool first = it.first(), codes = it.codes();
            const uint32_t b = pn % kDecPBufs, b2 = (pn + 1) % kDecPBufs;      // a bf16 tile's lo is in the second
            if (!warp_wait(&p_full[b], (pn / kDecPBufs) & 1, abort_flag)) break;
            if (!codes && !warp_wait(&p_full[b2], ((pn + 1) / kDecPBufs) & 1, abort_flag)) break;
            pn += codes ? 1 : 2;
            if (first && !warp_wait(o_empty, (it.item & 1) ^ 1, abort_flag)) break;
            tc_fence_after();
            const int nvalid = it.nvalid();
            const uint32_t p_base = smem_u32(sm + kQsP + b * kDecPBytes);
            const int per = codes ? 1 : 2;                 // slabs per 128-channel chunk
            const int step = codes ? 32 : 16;              // keys per MMA; steps without a key are left out
            const int steps = (nvalid + step - 1) / step;
            const int nz = (steps * step - nvalid) * 8;    // 16-byte chunks of rows in the last step without a key
            bool ok = true;
#pragma unroll 1
            for (int c = 0; c < 4; ++c, vs += per) {
                const uint32_t st = vs % kQdRing;          // per == 2: vs is even, the two slabs adjoin
                for (int x = 0; ok && x < per; ++x)
                    ok = warp_wait(&full_v[st + x], (vs / kQdRing) & 1, abort_flag);
                if (!ok) break;
                uint8_t* slab = sm + kQsV + st * kSlabBytes;
                if (nz > 0 && st == 0) {
                    // rows >= nvalid may hold anything (memory past the visible entries, ring slots not
                    // yet written): zero them in all four slabs so 0-probability keys contribute exactly 0
#pragma unroll 1
                    for (int x = per; ok && x < kQdRing; ++x) ok = warp_wait(&full_v[x], (vs / kQdRing) & 1, abort_flag);
                    if (!ok) break;
#pragma unroll 1
                    for (int sl = 0; sl < kQdRing; ++sl)
#pragma unroll 1
                        for (int i = lane; i < nz; i += 32)
                            *reinterpret_cast<uint4*>(slab + sl * kSlabBytes + nvalid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                const uint32_t dst = tmem + kQdO + 64 * c;
                const uint64_t vd = smem_desc_sw128(smem_u32(slab), kSlabBytes, 1024);
                const uint64_t p8 = smem_desc_sw64(p_base, 8192, 512), pw = smem_desc_sw128(p_base, 8192, 1024);
                const uint64_t pl = smem_desc_sw128(smem_u32(sm + kQsP + b2 * kDecPBytes), 8192, 1024);
                if (elect_one()) {
                    if (E8 && codes) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)     // 32 keys each
                            if (kk < steps) {
                                mma_f8(dst, vd + kk * (4096 >> 4), p8 + kk * (2048 >> 4), id_hi, (first && kk == 0) ? 0u : 1u);
                                mma_f8(dst, vd + kk * (4096 >> 4), p8 + ((8192 + kk * 2048) >> 4), id_lo, 1u);
                            }
                        mma_commit(&empty_v[st]);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)     // 16 keys each
                            if (kk < steps) {
                                mma_ss(dst, vd + kk * (2048 >> 4), pw + kk * (2048 >> 4), id_w, (first && kk == 0) ? 0u : 1u);
                                mma_ss(dst, vd + kk * (2048 >> 4), pl + kk * (2048 >> 4), id_w, 1u);
                            }
                        mma_commit(&empty_v[st]);
                        mma_commit(&empty_v[st + 1]);
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) {
                mma_commit(&p_empty[b]);
                if (!codes) mma_commit(&p_empty[b2]);
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
        // the two scale bytes of this thread's key in tile `tile` of the iterator's unit (1.0 for bf16 keys)
        auto scales = [&](int tile) -> uint32_t {
            const int j = tile * kDecTile + r;
            if (!E8 || it.done || j >= it.t.nc) return 0x7f7fu;
            long long row;
            if (PAGED)
                row = (long long)q_page(p, it.t.b, j, false) * p.page_size + j % p.page_size;
            else
                row = (long long)it.t.b * p.Nmax + j;
            return __ldg(p.sc + row * p.Hkv + it.t.g);
        };
        uint32_t sc = scales(it.tile);
        float lsum[32];       // this thread's share of the row sums, per head
#pragma unroll
        for (int h = 0; h < 32; ++h) lsum[h] = 0.f;
        // A wait of this warp ran out.  The warps leave together, at the barrier that every tile has; until then a
        // warp that gave up goes on without waiting for long (the abort flag is set).
        bool bad = false;
        uint32_t nq = 0, pn = 0;              // query operands, P buffers used
        // A piece's record is written behind the making of the next piece's query operand, whose products then run
        // beside it.
        int rec = -1, rec_item = 0;
        for (int n = 0;; ++n) {
            const bool first = it.first(), last = it.last(), codes = it.codes();
            if (!it.done && it.qfirst()) {
                softmax_bar();               // qs_s is no longer read
                // ---- the query operand: q (with QK normalisation q / rms(q) * g_q * g_k, since q_hat . k_hat =
                // (q' . k) / rms(k)), as two e4m3 terms for codes, else in bf16.  A warp makes one head at a time, in
                // place: the head's row of every slab is what its two 8-bit rows take.
                if ((NORM || codes) && !bad) {
                    bad = !warp_wait(q_tma, nq & 1, abort_flag);        // (an operand of garbage is never used then)
                    const int c0 = 16 * lane;                // this lane's channels
                    float g[NORM ? 16 : 1];
                    if (NORM) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 a = __ldg(reinterpret_cast<const float4*>(p.gq + c0 + e));
                            const float4 b2 = __ldg(reinterpret_cast<const float4*>(p.gk + c0 + e));
                            g[e] = a.x * b2.x;
                            g[e + 1] = a.y * b2.y;
                            g[e + 2] = a.z * b2.z;
                            g[e + 3] = a.w * b2.w;
                        }
                    }
#pragma unroll 2
                    for (int i = 0; i < 8; ++i) {
                        const int h = warp - kQdSoftWarp0 + kDecSoftWarps * i;
                        uint8_t* row = sm + kQsQ + Shape::q_tile(lane >> 2);
                        uint4* src0 = reinterpret_cast<uint4*>(row + sw128(h, 2 * (lane & 3)));
                        uint4* src1 = reinterpret_cast<uint4*>(row + sw128(h, 2 * (lane & 3) + 1));
                        const uint4 xa = *src0, xb = *src1;
                        const uint32_t w8[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
                        float f[16];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            f[2 * e] = bf16lo(w8[e]);
                            f[2 * e + 1] = bf16hi(w8[e]);
                        }
                        if (NORM) {
                            float ss = 0.f;
#pragma unroll
                            for (int e = 0; e < 16; ++e) ss = fmaf(f[e], f[e], ss);
                            ss = q_warp_sum(ss);
                            const float inv = rsqrtf(ss * (1.f / kDecD) + p.eps);
#pragma unroll
                            for (int e = 0; e < 16; ++e) f[e] *= inv * g[e];
                        }
                        if (E8 && codes) {
                            float am = 0.f;                  // (fmaxf leaves NaN out)
#pragma unroll
                            for (int e = 0; e < 16; ++e) am = fmaxf(am, fabsf(f[e]));
                            // non-negative floats are ordered as their bits
                            uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(am));
                            if (top == 0x7f800000u) {        // an infinity: it becomes NaN, and the rest sets the scale
                                am = 0.f;
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    am = fmaxf(am, q_mag(f[e]));
                                    f[e] = q_prep(f[e], 1.f);
                                }
                                top = __reduce_max_sync(0xffffffffu, __float_as_uint(am));
                            }
                            const uint32_t byte = q_scale_byte(__uint_as_float(top));
                            const float qi = q_inv_scale(byte);
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t l0, l1;
                                const uint32_t h0c = q_split(f[4 * e] * qi, f[4 * e + 1] * qi, l0);
                                const uint32_t h1c = q_split(f[4 * e + 2] * qi, f[4 * e + 3] * qi, l1);
                                hi[e] = h0c | h1c << 16;
                                lo[e] = l0 | l1 << 16;
                            }
                            __syncwarp();                    // every lane has read its part of the row
                            uint8_t* dst = sm + kQsQ + (lane >> 3) * Shape::kHi + sw128(h, lane & 7);
                            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                            *reinterpret_cast<uint4*>(dst + Shape::kLo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                            if (lane == 0) qs_s[h] = q_scale(byte) * p.scale_log2;
                        } else {
                            *src0 = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                               pack_bf16x2(f[6], f[7]));
                            *src1 = make_uint4(pack_bf16x2(f[8], f[9]), pack_bf16x2(f[10], f[11]), pack_bf16x2(f[12], f[13]),
                                               pack_bf16x2(f[14], f[15]));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_full);
                }
                ++nq;
                if (!codes && sidx < 64) qs_s[sidx] = p.scale_log2;
                softmax_bar();               // qs_s
            }

            if (rec >= 0) {
                if (!bad) bad = !warp_wait(o_full, rec_item & 1, abort_flag);
                tc_fence_after();
                float* orec = p.rec_o + ((size_t)rec * 64 + h0) * kDecD + r;
                const int hn = min(32, p.G - h0);        // heads of this half
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float o[32];
                    tmem_ld32(tmem + lane_off + kQdO + 64 * c + h0, o);
                    tmem_wait_ld32(o);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < hn) orec[(size_t)j * kDecD + 128 * c] = o[j];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_empty);
                rec = -1;
            }
            if (it.done) break;
            const int sb = n % look;
            const bool valid = r < it.nvalid();
            const uint32_t sc_next = last ? 0u : scales(it.tile + 1);      // loaded while this tile is worked on
            if (!bad) bad = !warp_wait(&s_full[sb], (n / look) & 1, abort_flag);
            tc_fence_after();
            float kscale = q_scale(sc & 0xffu);
            if (NORM) {                      // (ahead of the logits: both at once would not fit the registers)
                float d[32];
                tmem_ld32(tmem + lane_off + kQdKK + q4 * 32, d);
                tmem_wait_ld32(d);
                float diag = 0.f;
#pragma unroll
                for (int j = 0; j < 32; ++j) diag = (j == lane) ? d[j] : diag;
                kscale *= rsqrtf(diag * (1.f / kDecD) * kscale * kscale + p.eps);
            }
            float z[32];
            tmem_ld32(tmem + lane_off + 64 * sb + h0, z);
            tmem_wait_ld32(z);
            if (joined && codes) {           // the share of q lo
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float zl[16];
                    tmem_ld16(tmem + lane_off + 64 * sb + 64 + h0 + 16 * c, zl);
                    tmem_wait_ld16(zl);
#pragma unroll
                    for (int h = 0; h < 16; ++h) z[16 * c + h] += zl[h];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[sb]);
            // y = logit + log2(vscale)
            const float lv = (float)((int)(sc >> 8) - 127);
            const float rv = q_inv_scale(sc >> 8);
            bool need = first;
#pragma unroll
            for (int h = 0; h < 32; h += 4) {
                const float4 qs = *reinterpret_cast<const float4*>(qs_s + h0 + h);
                const float4 mm = *reinterpret_cast<const float4*>(m_s + h0 + h);
                z[h] = valid ? fmaf(z[h] * kscale, qs.x, lv) : -INFINITY;
                z[h + 1] = valid ? fmaf(z[h + 1] * kscale, qs.y, lv) : -INFINITY;
                z[h + 2] = valid ? fmaf(z[h + 2] * kscale, qs.z, lv) : -INFINITY;
                z[h + 3] = valid ? fmaf(z[h + 3] * kscale, qs.w, lv) : -INFINITY;
                need |= (z[h] > mm.x + thr) | (z[h + 1] > mm.y + thr) | (z[h + 2] > mm.z + thr) | (z[h + 3] > mm.w + thr);
            }

            // ---- reference m (shared m_s[64]): the first tile's maximum, then only when some y
            // exceeds it by thr
            if (softmax_any(need || bad)) {
                if (softmax_any(bad)) break;
                const float tmax = colreduce32<true>(z, lane);
                red[q4 * 64 + h0 + lane] = tmax;
                softmax_bar();
                if (sidx < 64) {
                    const float mo = first ? -INFINITY : m_s[sidx];
                    const float mt = fmaxf(fmaxf(red[sidx], red[64 + sidx]), fmaxf(red[128 + sidx], red[192 + sidx]));
                    // held finite: keys of logit -inf then weigh nothing beside later ones, and NaN stays in the sums
                    const float mn = fmaxf(fmaxf(mo, mt - shift), kLowest);
                    al_s[sidx] = first ? 0.f : ex2(mo - mn);
                    m_s[sidx] = mn;
                }
                softmax_bar();
                if (!first) {
#pragma unroll
                    for (int h = 0; h < 32; ++h) lsum[h] *= al_s[h0 + h];
                    // rescale O^T once the previous PV has landed
                    bad = !warp_wait(&p_empty[(pn - 1) % kDecPBufs], ((pn - 1) / kDecPBufs) & 1, abort_flag);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        const uint32_t ta = tmem + lane_off + kQdO + 64 * c + h0;
                        tmem_ld32(ta, o);
                        tmem_wait_ld32(o);
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(o[j] * al_s[h0 + j]);
                        tmem_st16(ta, w);
                        tmem_st16(ta + 16, w + 16);
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
            const uint32_t b = pn % kDecPBufs, b2 = (pn + 1) % kDecPBufs;
            if (!bad) bad = !warp_wait(&p_empty[b], ((pn / kDecPBufs) & 1) ^ 1, abort_flag);
            if (!bad && !codes) bad = !warp_wait(&p_empty[b2], (((pn + 1) / kDecPBufs) & 1) ^ 1, abort_flag);
            uint8_t* pt = sm + kQsP + b * kDecPBytes;
            if (!bad) {
                if (E8 && codes) {
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
                    for (int c = 0; c < 4; ++c) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a0 = z[8 * c + 2 * e], a1 = z[8 * c + 2 * e + 1];
                            hi[e] = pack_bf16x2(a0, a1);
                            lo[e] = pack_bf16x2(a0 - bf16lo(hi[e]), a1 - bf16hi(hi[e]));
                        }
                        *reinterpret_cast<uint4*>(pt + sw128(r, 4 * hh + c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(sm + kQsP + b2 * kDecPBytes + sw128(r, 4 * hh + c)) =
                            make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&p_full[b]);
                    if (!codes) mbar_arrive(&p_full[b2]);
                }
            }
            pn += codes ? 1 : 2;

            if (last) {
                // ---- end of this CTA's piece of unit u: the row sums over all key rows for its record
                // (reference, sum, unnormalised O^T)
                const int u = it.u;
                rec = cta + u;
                rec_item = it.item;
                const float tsum = colreduce32<false>(lsum, lane);
                red[q4 * 64 + h0 + lane] = tsum;
                softmax_bar();
                if (sidx == 0) {
                    if (it.tb == 0) p.meta[2 * u] = cta;
                    if (it.tend == it.ntiles) p.meta[2 * u + 1] = cta;
                }
                if (sidx < 64) {
                    p.rec_m[(size_t)rec * 64 + sidx] = m_s[sidx];
                    p.rec_l[(size_t)rec * 64 + sidx] = (red[sidx] + red[64 + sidx]) + (red[128 + sidx] + red[192 + sidx]);
                }
                softmax_bar();     // red[] is free again before the next piece's first reduction
#pragma unroll
                for (int h = 0; h < 32; ++h) lsum[h] = 0.f;
            }
            it.next();
            sc = last ? scales(it.tile) : sc_next;
        }
    }

    __syncwarp();      // every role reconverges its warp before the CTA-wide barrier
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // the merge follows this pass: its end is the prefix pass's end too
    if (p.pfx_total > 0 && cta == 0 && threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace hca
