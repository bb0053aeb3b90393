// Causal prefill attention over E4M3 caches with a scale per block and KV head.
//
// What it computes, its work items, their order and splits, and its schedule are those
// of pkv_prefill_wide.cuh (128-key tiles, one score buffer per query tile, P over S in
// two halves, the MMA warps' lock).  What differs:
//
//  * Scores run on the E4M3 path with K as the raw codes, so a K tile is half the bytes
//    and nobody converts it.  Q becomes two E4M3 parts, q = sq (high + low), once per
//    item and row: two multiplications at twice the rate of bf16's one, in the same
//    shared memory.  A key's multiplier inside the exponential is the softmax scale times
//    its row's sq times its 16-token box's K scale: no score is scaled on its own.
//  * V's codes become f16, times f = their block's scale over a unit in which O is held, in
//    buffers of their own (they are twice the codes' bytes).  With scales that are powers
//    of two that product is exact, f being kept within [2^-15, 2^7] (codes end at 2^-9, f16
//    at 2^-24).  The unit, a power of two, moves where a tile's largest scale leaves
//    [2^-2, 2^7) of it; O is then rescaled with the running maximum.  Of a scale below
//    2^-15 units the rest, g = 2^-1, 2^-2, ..., joins the weights: its scores are moved by
//    log2 g before the running maximum sees them, P holds w g, and the sum gets its
//    w = (w g) / g.  So a row whose weight lies on a block of small scale keeps it, whatever
//    the other blocks hold.  Rows that see no larger block of such a tile (it is in their
//    future) hold O in a unit of their own.  A tile with such a block costs two more loops
//    over its scores (all of them, ragged prompts in blocks of 16: 280 -> 631 us); no other
//    tile knows of it.
//  * A NaN in V's codes would reach every row of its item through a weight of 0 (the rows
//    that do not see its token).  Nothing looks for one but an item's end, where an element
//    of O is NaN and the row's sum is not: the item is then done again, the producer taking
//    NaN out of its codes a tile behind the copies, and NaN written where a row sees one.
//    (Codes looked at as they are converted: 16k 253, ragged 283, long chunk 773 us; so 251,
//    280, 760.  With a NaN in each sequence's first block 750, 830, 1820; with clean codes
//    loaded by the producer itself 1120, 1150, 3140.)
//  * The producer, whose time is free, does what can be done once per tile: it loads
//    each box's block two tiles ahead and its scales one, works out V's factors and the
//    unit, and waits for V's f16 buffer, so that a softmax warp waits once per tile for
//    all of that (each wait, met or not, is 100 to 180 cycles of its chain).
//  * The instructions of a tile are few: the main path has no masks (a short loop writes
//    -inf into the scores of the tiles that have some) and no second form for boxes of
//    different scales, and the halves of a row's exponentials share theirs.  With forms
//    for each, 32 KB of instructions, the warps waited for those: 815 -> 747 us below,
//    394 -> 277 us for ragged prompts.
//
// Precision: Q's parts below; P and V in f16, fp32 sums.  Where V's scales of a tile lie
// within 2^13 of each other, V is exact for powers of two (else rounded twice, 2^-11 each)
// and w rounded by 2^-11 of itself or 2^-25 of the row's largest.  Elsewhere w g is, by
// 2^-11 of itself or 2^-25 of the row's largest w g.
//
// Measured: 8 sequences of 2048 new tokens on up to 2048 (16 heads, 275 GFLOP) 251 us,
// 1095 TFLOP/s, tensor pipe 49% busy; one chunk of 2048 on 28672 (32 heads, 996 GFLOP)
// 760 us, 1310 TFLOP/s, 60%.  Bound by the chain of a query tile (scores, maximum,
// exponentials, P.V, next scores: some 3000 cycles per 128 keys against 2048 of MMA), and
// where items are short by their ends: Q's conversion 3600 cycles, the output 2200.
// Not kept: sixteen softmax warps, with half of a row each (bookkeeping per warp: 962 us
// for the chunk, 850 at the time); four warps for the conversions (1100, 996 at the
// time); the lock passed on before the wait for P.V (774), or left out (816); 96 of a
// row's 128 scores kept in registers (1048: instructions).
//
// Warps (352 threads): 0..3 softmax of query tile A, 4..7 of tile B (thread = row = TMEM
// lane); 8 producer; 9, 10 the MMAs of tiles A and B.  TMEM as in pkv_prefill_wide.cuh.
// Shared memory (D = 128): Q 64 KB, two stages each of K and V codes, 16 KB each, three
// buffers of V as f16, 32 KB each.
#pragma once

#include "pkv_prefill_wide.cuh"

namespace pkv {

constexpr int kSKeys = kWKeys;  // keys per tile
constexpr int kSKStages = 2;    // K ring: codes
constexpr int kSRStages = 2;    // V ring: codes
constexpr int kSVStages = 3;    // V as f16: one more than a tile's P.V of both query tiles needs
                                // (with two, a query tile that is ahead waits for the other)
// Tiles whose scales are kept: a tile's are read (K's) until the warp has its P, by which
// time it has not yet taken the V codes of the tile after the next; the producer goes on
// to a fourth after that.
constexpr int kSScales = 4;
static_assert(kSScales >= kSRStages + 2, "a tile's scales outlive its stage");
// q_full[2], q_conv[2], q_empty[2], k_full, k_empty [kSKStages] each, r_full, r_empty
// [kSRStages] each, v_conv, v_empty [kSVStages] each, per query tile s_full,
// pv_ready[2 halves], pv_done, o_free, then item_ready[2], item_free[2], mma_done, raw[2]
constexpr int kSBars = 6 + 2 * kSKStages + 2 * kSRStages + 2 * kSVStages + 10 + 4 + 1 + 2;

// What the softmax warps need of a key tile beside its codes; the producer brings it with
// V's.  read: which of the eight boxes are read (a bit each), above them which have a scale
// that is NaN, and kFarApart.  k: their K scales (1 where there is none).  V's scales are `unit` f g: v = f, as pairs of f16, and lg = log2 g,
// 0 but in tiles with kFarApart.
constexpr int kFarApart = 0x10000;
struct __align__(16) TileScales {
    float k[kSKeys / kBox];
    uint32_t v[kSKeys / kBox];
    float lg[kSKeys / kBox];
    int read;
    float unit;
    int pad[2];
};

struct ScaledSmem {
    size_t q, k, r, v, scales, bars, items, nans, slot, total;
};

__host__ __device__ inline ScaledSmem scaled_smem_layout(int D)
{
    ScaledSmem L;
    size_t o = 0;
    L.q = o;  // [tile][D/64 halves][128 rows][128 B]
    o += (size_t)2 * (D / 64) * kTcRows * 128;
    L.k = o;  // stages of [128 keys][D codes]
    o += (size_t)kSKStages * kSKeys * D;
    L.r = o;  // alike, V
    o += (size_t)kSRStages * kSKeys * D;
    L.v = o;  // stages of [D/64 halves][128 keys][128 B]
    o += (size_t)kSVStages * (D / 64) * kSKeys * 128;
    L.scales = o;  // of the last kSScales tiles
    o += kSScales * sizeof(TileScales);
    L.bars = o;
    o += 8 * kSBars;
    L.items = align_up(o, 16);  // two published work items
    o = L.items + 2 * sizeof(WideItem);
    L.nans = o;  // of the two items: whether it has to be done again, then per column the
    o += 2 * (1 + D) * sizeof(int);  // first token (of the sequence) whose V is NaN
    o = align_up(o, 16);
    L.slot = o;  // TMEM base, and the MMA warps' lock
    o += 16;
    L.total = align_up(o, 16) + 1024;
    if (L.total < kTcMinSmem)
        L.total = kTcMinSmem;
    return L;
}

// Eight words, 32 bytes.
__device__ __forceinline__ void store32(void *to, const uint32_t *v, bool aligned32)
{
    if (aligned32) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        uint4 *d = reinterpret_cast<uint4 *>(to);
        d[0] = make_uint4(v[0], v[1], v[2], v[3]);
        d[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// 2^e of a whole e within [-126, 127].
__device__ __forceinline__ float exp2_int(float e) { return __uint_as_float((uint32_t)(127 + (int)e) << 23); }

// a / b for powers of two whose quotient is within that range.
__device__ __forceinline__ float exp2_ratio(float a, float b)
{
    return __uint_as_float(0x3f800000u + __float_as_uint(a) - __float_as_uint(b));
}

// Eight E4M3 codes times f (a pair of f16) as eight f16.
__device__ __forceinline__ uint4 e4m3x8_to_f16(uint32_t a, uint32_t b, uint32_t f)
{
    uint4 r;
    e4m3x4_to_f16x2x2(a, r.x, r.y);
    e4m3x4_to_f16x2x2(b, r.z, r.w);
    r.x = f16x2_mul(r.x, f);
    r.y = f16x2_mul(r.y, f);
    r.z = f16x2_mul(r.z, f);
    r.w = f16x2_mul(r.w, f);
    return r;
}

// O (a row per thread) times a number per row.  In place while P . V rests: S_t(j) was
// issued after P.V_t(j - 1) completed, and the next P.V waits for this group's P.
template <int D> __device__ __forceinline__ void rescale_o(uint32_t tO, float by)
{
#pragma unroll 1
    for (int cc = 0; cc < D / 32; cc++) {
        uint32_t ro[32];
        tc::ld32(tO + 32 * cc, ro);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i++)
            ro[i] = __float_as_uint(__uint_as_float(ro[i]) * by);
        tc::st32(tO + 32 * cc, ro);
    }
    tc::wait_st();
}

// A row's running maximum and sum, the unit of the tile at hand and the one its O is in.
struct RowState {
    float m, l, unit, o_unit;
};

// What a tile asks of its scores (masked ones are -inf already) where it has scales that
// are NaN or V's far apart.  NaN: into the scores that are seen in their boxes.  Far apart:
// log2 g joins the scores, 2^shift g in a unit of the row's own; the running maximum follows
// at once, so that the sum, which is of w, can be given the (w g) / g - w g that it lacks
// when w g is added to it.  lim: the last key of the tile that the row sees.  Out of line,
// for the instructions of what always runs barely fit the caches (inline ragged 278 us, long
// chunk 769; so 274, 761).
template <int D>
__device__ __noinline__ RowState odd_scales(uint32_t tS, uint32_t tO, const TileScales &ts, uint32_t boxes, int lim,
                                            float sl, RowState s, bool has_o)
{
    constexpr int kBoxes = kSKeys / kBox;
    uint32_t r[16];
#pragma unroll 1
    for (int b = 0; b < kBoxes; b++) {
        if (!((boxes >> (kBoxes + b)) & 1u))
            continue;
        tc::ld16(tS + kBox * b, r);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < kBox; i++)
            r[i] = kBox * b + i > lim ? r[i] : 0x7fffffffu;
        tc::st16(tS + kBox * b, r);
    }
    tc::wait_st();
    if (!(boxes & kFarApart))
        return s;
    float seen = -INFINITY;
#pragma unroll 1
    for (int b = 0; b < kBoxes; b++)
        if (((boxes >> b) & 1u) && lim >= kBox * b && ts.v[b])
            seen = fmaxf(seen, ts.lg[b]);
    const float shift = seen > -INFINITY ? -seen : 0.f;
    s.unit *= exp2_int(-shift);
    float mn = s.m;
#pragma unroll 1
    for (int b = 0; b < kBoxes; b++) {
        const float c = sl * ts.k[b], move = (ts.lg[b] + shift) / c;
        tc::ld16(tS + kBox * b, r);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < kBox; i++) {
            const float moved = __uint_as_float(r[i]) + move;
            mn = fmaxf(mn, moved * c);
            r[i] = __float_as_uint(moved);
        }
        tc::st16(tS + kBox * b, r);
    }
    tc::wait_st();
    const float alpha = mn == -INFINITY ? 1.f : fast_exp2(s.m - mn);
    if (has_o)
        rescale_o<D>(tO, alpha * exp2_ratio(s.o_unit, s.unit));
    s.o_unit = s.unit;
    s.m = mn;
    s.l *= alpha;
    const float nm = mn == -INFINITY ? 0.f : -mn;
#pragma unroll 1
    for (int b = 0; b < kBoxes; b++) {
        tc::ld16(tS + kBox * b, r);
        tc::wait_ld();
        const float c = sl * ts.k[b];
        float e = 0.f;
#pragma unroll
        for (int i = 0; i < kBox; i++)
            e += fast_exp2(fmaf(__uint_as_float(r[i]), c, nm));
        s.l = fmaf(exp2_int(-ts.lg[b] - shift) - 1.f, e, s.l);
    }
    return s;
}

// NaN in a tile of V's codes (of `keys` tokens; those of boxes that are not read are cleared as
// they are converted): 0 in their place, their token noted for their column.
template <int D>
__device__ __noinline__ void clean_codes(uint8_t *tile, uint32_t read, int key0, int keys, int *nan_from, int lane)
{
    constexpr int kPieces = D / 16;
#pragma unroll 8
    for (int i = lane; i < kSKeys * kPieces; i += 32) {
        const int r = i / kPieces;
        uint4 *at = reinterpret_cast<uint4 *>(tile) + i;
        const uint4 w = *at;
        const auto nan = [](uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
        if (!(nan(w.x) | nan(w.y) | nan(w.z) | nan(w.w)) || r >= keys || !((read >> (r / kBox)) & 1u))
            continue;
        // swizzled as it was copied
        const int piece = D == 128 ? i % kPieces ^ (r & 7) : i % kPieces ^ ((r >> 1) & 3);
        uint32_t *words = reinterpret_cast<uint32_t *>(at);
#pragma unroll 1
        for (int c = 0; c < 4; c++) {
            uint32_t t = nan(words[c]);  // the top bit of a byte that is
            words[c] &= ~((t >> 7) * 0xffu);
            for (; t; t &= t - 1)
                atomicMin(nan_from + 16 * piece + 4 * c + (__ffs(t) >> 3) - 1, key0 + r);
        }
    }
    fence_proxy_async_smem();  // the next copy into the stage is behind this
    __syncwarp();
}

// NaN into the columns of an output row that see one.
template <int D, typename T> __device__ __noinline__ void write_nans(T *out, T nan, const int *nan_from, int pos)
{
#pragma unroll 1
    for (int d = 0; d < D; d++)
        if (nan_from[d] <= pos)
            out[d] = nan;
}

// SPLIT: p.splits > 1.  Of its own, for the others' items are 4% slower with it
// where they are short.
template <int D, int G, bool SPLIT>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_prefill_scaled_kernel(const __grid_constant__ CUtensorMap tmq,
                              const __grid_constant__ CUtensorMap tmk,
                              const __grid_constant__ CUtensorMap tmv, const PrefillParams p)
{
    constexpr int TPC = kTcRows / G;               // query tokens per tile
    constexpr int HALVES = D / 64;
    constexpr uint32_t kQHalf = kTcRows * 128;     // 16 KB
    constexpr uint32_t kQTile = HALVES * kQHalf;
    constexpr uint32_t kTile = kSKeys * D;         // one K (or V) tile of codes
    constexpr uint32_t kVHalf = kSKeys * 128;      // 64 columns of a V tile as f16
    constexpr uint32_t kVTile = HALVES * kVHalf;
    constexpr int kBoxes = kSKeys / kBox;          // 16-token boxes per tile
    constexpr unsigned FULL = 0xffffffffu;
    constexpr float kLazy = 8.f;
    const int splits = SPLIT ? p.splits : 1, whole = SPLIT ? p.whole : 0;
    const long long units = SPLIT ? whole + (long long)(p.n_items - whole) * splits : p.n_items;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const ScaledSmem L = scaled_smem_layout(D);
    uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + L.bars);  // [2] Q tile t landed
    uint64_t *q_conv = q_full + 2;                // [2] ... and became E4M3 parts (4 warps)
    uint64_t *q_empty = q_conv + 2;               // [2] tile t's last S of the item completed (4 warps)
    uint64_t *k_full = q_empty + 2;
    uint64_t *k_empty = k_full + kSKStages;       // both tiles' S of the K tile completed (4 warps each)
    uint64_t *r_full = k_empty + kSKStages;       // V codes landed
    uint64_t *r_empty = r_full + kSRStages;       // ... and were read (8 warps)
    uint64_t *v_conv = r_empty + kSRStages;       // the V tile as f16 (8 warps)
    uint64_t *v_empty = v_conv + kSVStages;       // both tiles' P.V of the V tile completed
    uint64_t *s_full = v_empty + kSVStages;       // [2] S_t written
    uint64_t *pv_ready = s_full + 2;              // [half of the keys][2] P_t written (4 warps)
    uint64_t *pv_done = pv_ready + 4;             // [2] P.V_t completed
    uint64_t *o_free = pv_done + 2;               // [2] O_t read out by its epilogue (4 warps)
    uint64_t *item_ready = o_free + 2;            // [2] item parameters published
    uint64_t *item_free = item_ready + 2;         // [2] ... no longer needed
    uint64_t *mma_done = item_free + 2;           // every MMA of the CTA completed
    uint64_t *raw = mma_done + 1;                 // [2] V codes landed that are to be looked through
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem + L.slot);
    const Turn turn{slot + 1};
    WideItem *items = reinterpret_cast<WideItem *>(smem + L.items);
    uint8_t *sQ = smem + L.q, *sK = smem + L.k, *sR = smem + L.r, *sV = smem + L.v;
    TileScales *scales = reinterpret_cast<TileScales *>(smem + L.scales);
    int *again = reinterpret_cast<int *>(smem + L.nans);  // [2]
    int *nan_from = again + 2;                            // [2][D]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_launch_dependents();
    if (warp == kTcProducerWarp && lane == 0) {
        for (int t = 0; t < 2; t++) {
            mbar_init(&q_full[t], 1);
            mbar_init(&q_conv[t], 4);
            mbar_init(&q_empty[t], 4);
            mbar_init(&s_full[t], 1);
            mbar_init(&pv_ready[t], 4);
            mbar_init(&pv_ready[2 + t], 4);
            mbar_init(&pv_done[t], 1);
            mbar_init(&o_free[t], 4);
            mbar_init(&item_ready[t], 1);
            mbar_init(&item_free[t], 10);  // two MMA warps, eight softmax warps
        }
        for (int s = 0; s < kSKStages; s++) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 8);
        }
        for (int s = 0; s < kSRStages; s++) {
            mbar_init(&r_full[s], 1);
            mbar_init(&r_empty[s], 8);
        }
        for (int s = 0; s < kSVStages; s++) {
            mbar_init(&v_conv[s], 8);
            mbar_init(&v_empty[s], 2);  // both MMA warps
        }
        mbar_init(mma_done, 2);
        mbar_init(&raw[0], 1);
        mbar_init(&raw[1], 1);
        *turn.word = 0;
        again[0] = again[1] = 0;
        fence_mbarrier_init();
    } else if (warp == kTcMmaWarp) {
        tc::alloc(smem_u32(slot), kTcCols);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *slot;
    const int nC = (int)gridDim.x;
    const int c = (int)blockIdx.x;

    if (warp == kTcProducerWarp) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tensormap(&tmq);
            prefetch_tensormap(&tmk);
            prefetch_tensormap(&tmv);
        }
        grid_dependency_wait();  // K/V may have just been written by store_kvcache
        int gk = 0, gv = 0;       // K and V tiles issued so far (all items)
        int gr = 0, gc = 0;       // V tiles to look through: issued, and done
        int q_loads[2] = {0, 0};  // Q tiles A and B loaded so far
        bool ok = true;
        int n = 0;                // items published
        int k = 0;                // walk rounds
        for (;;) {
            // ---- slot n & 1, once the item two back is done with it
            const int sl = n & 1;
            if (n >= 2 && !__all_sync(FULL, mbar_wait_asleep(&item_free[sl], ((n >> 1) & 1) ^ 1))) {
                ok = false;
                break;  // the other warps time out on item_ready and stop
            }
            // ---- that item again, if its V held NaN; else the next item with work (round k:
            // forward, then backward), or the end
            WideItem item{{-1, 0, 0, 0, 0, 0, {0, 0}}, 0, 0, 0, 0};
            PrefillItem &it = item.f;
            bool repeat = again[sl] != 0;
            for (; !repeat; k++) {
                const long long at = (long long)k * nC + ((k & 1) ? nC - 1 - c : c);
                if (at >= units)
                    break;
                // the split items' first pieces, then their second ones: items that turn
                // out too short to be split fill the SMs like any others
                int pos = (int)at, piece = -1;
                if (SPLIT && at >= whole) {
                    piece = ((int)at - whole) / (p.n_items - whole);
                    pos -= piece * (p.n_items - whole);
                }
                const PrefillWork w = p.B <= 32 ? prefill_schedule<2 * TPC, 1>(p, lane, pos)
                                                : prefill_schedule<2 * TPC, kSchedChunks>(p, lane, pos);
                int cq0 = w.cq0, cq1 = w.cq1, ck0 = w.ck0, ck1 = w.ck1;
                if (w.b >= 0 && cq0 == kNotLoaded) {
                    cq0 = __ldg(p.cu_q + w.b);
                    cq1 = __ldg(p.cu_q + w.b + 1);
                    ck0 = __ldg(p.cu_k + w.b);
                    ck1 = __ldg(p.cu_k + w.b + 1);
                }
                const bool sane = w.b >= 0 && prefill_seq_sane(p, cq0, cq1, ck0, ck1);
                if (w.b >= 0 && !sane && lane == 0)
                    flag_error(p.err_flag, 0x4 /* PKV_FLAG_BAD_CONTEXT_LEN */);
                const int tok0 = w.tile * 2 * TPC;
                if (sane && tok0 < cq1 - cq0) {
                    it.kvh = w.kvh;
                    it.tok0 = tok0;
                    it.cq0 = cq0;
                    it.q_len = cq1 - cq0;
                    it.k_len = ck1 - ck0;
                    const int base = it.k_len - it.q_len;
                    it.nkt[0] = (base + min(it.q_len, tok0 + TPC) - 1) / kSKeys + 1;
                    it.nkt[1] = tok0 + TPC < it.q_len
                                    ? (base + min(it.q_len, tok0 + 2 * TPC) - 1) / kSKeys + 1
                                    : 0;
                    if constexpr (SPLIT)
                        item.split = -1;
                    if (SPLIT && piece >= 0) {
                        const int nkt = max(it.nkt[0], it.nkt[1]);
                        const int chunk = wide_chunk(nkt, splits, p.least);
                        item.j0 = piece * chunk;
                        if (item.j0 >= nkt)
                            continue;  // the item has fewer splits
                        if (nkt > chunk) {
                            item.split = piece;
                            for (int t = 0; t < 2; t++)
                                it.nkt[t] = min(max(it.nkt[t] - item.j0, 0), chunk);
                        }
                    }
                    it.b = w.b;
                    k++;
                    break;
                }
                // up to kSchedMaxSeqs sequences, ranks are longest first, so
                // the first empty item ends this CTA's work (but for further pieces)
                if (!SPLIT && p.B <= kSchedMaxSeqs && w.b < 0) {
                    k = 0x3fffffff;
                    break;
                }
            }
            // ---- before the end, the last item may ask for it too
            int from = sl;
            if (!repeat && it.b < 0 && n >= 1) {
                from = sl ^ 1;
                if (!(ok = __all_sync(FULL, mbar_wait_asleep(&item_free[from], ((n - 1) >> 1) & 1))))
                    break;
                repeat = again[from] != 0;
            }
            if (repeat) {
                item = items[from];
                item.clean = 1;
#pragma unroll 1
                for (int d = lane; d < D; d += 32)
                    nan_from[sl * D + d] = 0x7fffffff;
            }
            __syncwarp();
            // ---- publish it
            if (lane == 0) {
                if (repeat)
                    again[from] = 0;
                items[sl] = item;
                mbar_arrive(&item_ready[sl]);
            }
            __syncwarp();
            if (it.b < 0)
                break;
            // ---- Q tiles, each once its tile's last S of the previous item completed
            for (int t = 0; t < 2 && ok; t++) {
                if (it.nkt[t] == 0)
                    continue;
                if (n >= 1 && !(ok = __all_sync(FULL, mbar_wait_asleep(&q_empty[t], (n - 1) & 1))))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&q_full[t], HALVES * kQHalf);
#pragma unroll
                    for (int h = 0; h < HALVES; h++)
                        tma_load_4d(sQ + t * kQTile + h * kQHalf, &tmq, 0, h, it.kvh * G,
                                    it.cq0 + it.tok0 + t * TPC, &q_full[t]);
                }
                ++q_loads[t];
            }
            if (!ok)
                break;
            n++;
            // ---- K and V tiles through their rings, in the order in which stages come free.
            // Lanes 0-7 resolve one 16-token box each: its block two tiles ahead of the
            // copies, the block's scales one tile ahead.
            const int nkt = max(it.nkt[0], it.nkt[1]);
            const int j0 = SPLIT ? item.j0 : 0;
            const int32_t *table = p.block_tables + (size_t)it.b * p.MBS;
            auto entry = [&](int j) -> int {
                const int key0 = (j0 + j) * kSKeys + lane * kBox;
                return (lane < kBoxes && j < nkt && key0 < it.k_len) ? __ldg(table + key0 / p.bs) : -1;
            };
            // (written by the store, maybe while this kernel was starting)
            auto scale_of = [&](const float *scales_of, int blk) {
                return blk >= 0 && blk < p.NB ? ld_gpu(scales_of + (size_t)blk * p.Hkv + it.kvh) : 0.f;
            };
            int blk = entry(0), blk_next = entry(1);
            float sk = scale_of(p.k_scales, blk), sv = scale_of(p.v_scales, blk);
            const int per = p.copy_rows;  // tokens per copy: so many lie in one block
            // V tiles' unit, 2^(unit - 127): moves to 2^-2 of a tile's largest scale where
            // that is not below 2^7 units (448 * 2^7 is within f16) or below 2^-2 (2^13 above
            // the least f)
            int unit = 127;
            for (int j = 0; j < nkt; j++) {
                const int key0 = (j0 + j) * kSKeys + lane * kBox;
                int row = -1;
                if (lane < kBoxes && key0 < it.k_len) {
                    if (blk >= 0 && blk < p.NB)
                        row = blk * p.bs + key0 % p.bs;
                    else
                        flag_error(p.err_flag, 0x2 /* PKV_FLAG_BAD_BLOCK */);
                }
                const uint32_t read = __ballot_sync(FULL, row >= 0);
                // A scale that is none (NaN) makes NaN the rows that see its box and no others,
                // so it goes into their scores, and what stands here is harmless.  (A masked
                // score is -inf, which no K scale may turn into NaN: zero neither.)
                const bool scaled = row >= 0 && sk >= 0.f && sk < INFINITY && sv >= 0.f && sv < INFINITY;
                const uint32_t broken = read & ~__ballot_sync(FULL, scaled);
                const float k = !scaled ? 1.f : sk == 0.f ? 0x1p-40f : sk;
                const uint32_t bits = scaled && sv > 0.f ? __float_as_uint(sv) : 0u;
                const int most = (int)(__reduce_max_sync(FULL, bits) >> 23);
                if (most > 0 && (j == 0 || most - unit >= 7 || most - unit < -2))
                    unit = max(most - 2, 1);
                const int e = bits ? (int)(bits >> 23) - unit : 0;
                const float f =
                    bits ? __uint_as_float((bits & 0x7fffffu) | (uint32_t)(127 + max(e, -15)) << 23) : 0.f;
                const uint32_t factor = pack_f16x2(f, f);
                const int lg = min(e + 15, 0), least = __reduce_min_sync(FULL, lg);
                // the next tile's, whose loads run while this one's stages are waited for
                blk = blk_next;
                sk = scale_of(p.k_scales, blk);
                sv = scale_of(p.v_scales, blk);
                blk_next = entry(j + 2);
                // rows past k_len of a run come along: their scores are masked and
                // their V rows zeroed
                const bool copies = row >= 0 && (lane * kBox) % per == 0;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(FULL, copies)) * per * D;
                const int at = lane * (kBox * D);
                const int rs = gv % kSRStages, vs = gv % kSVStages, ks = gk % kSKStages;
                ok = __all_sync(FULL, mbar_wait_asleep(&k_empty[ks], ((gk / kSKStages) & 1) ^ 1));
                if (!ok)
                    break;
                if (lane == 0)
                    mbar_arrive_expect_tx(&k_full[ks], bytes);
                __syncwarp();
                if (copies)
                    tma_load_3d(sK + (size_t)ks * kTile + at, &tmk, 0, it.kvh, row, &k_full[ks]);
                gk++;
                // V: its codes' stage, and the f16 buffer that they go to, so that the
                // softmax warps wait for the codes alone
                ok = __all_sync(FULL, mbar_wait_asleep(&r_empty[rs], ((gv / kSRStages) & 1) ^ 1) &&
                                          mbar_wait_asleep(&v_empty[vs], ((gv / kSVStages) & 1) ^ 1));
                if (!ok)
                    break;
                TileScales &ts = scales[gv % kSScales];
                if (lane < kBoxes) {
                    ts.k[lane] = k;
                    ts.v[lane] = factor;
                    // (a block of zeros has the least one, so that its weights are not the
                    // larger ones of a row in a unit of its own)
                    ts.lg[lane] = (float)(bits ? lg : least);
                }
                if (lane == 0) {
                    ts.read = (int)(read | broken << 8) | (least < 0 ? kFarApart : 0);
                    ts.unit = __uint_as_float((uint32_t)unit << 23);
                }
                __syncwarp();
                uint64_t *landed = item.clean ? &raw[gr & 1] : &r_full[rs];
                if (lane == 0)
                    mbar_arrive_expect_tx(landed, bytes);
                __syncwarp();
                if (copies)
                    tma_load_3d(sR + (size_t)rs * kTile + at, &tmv, 0, it.kvh, row, landed);
                if (__builtin_expect(item.clean, 0)) {
                    // the tile before while this one is on its way; the last one at once
                    gr++;
                    for (; gc < gr - (j + 1 < nkt); gc++) {
                        const int back = gr - 1 - gc, g = gv - back;
                        if (!(ok = __all_sync(FULL, mbar_wait_asleep(&raw[gc & 1], (gc >> 1) & 1))))
                            break;
                        const int first = (j0 + j - back) * kSKeys;
                        clean_codes<D>(sR + (size_t)(g % kSRStages) * kTile, scales[g % kSScales].read, first,
                                       it.k_len - first, nan_from + sl * D, lane);
                        if (lane == 0)
                            mbar_arrive(&r_full[g % kSRStages]);
                    }
                    if (!ok)
                        break;
                }
                gv++;
            }
            if (!ok)
                break;  // the other warps time out on their barriers and stop
        }
        if (lane == 0) {
            if (!ok)
                flag_error(p.err_flag, 0x8 /* PKV_FLAG_TIMEOUT */);
            // copies still in flight land before the CTA may exit
            for (int t = 0; t < 2; t++)
                if (q_loads[t] >= 1)
                    mbar_wait_asleep(&q_full[t], (q_loads[t] - 1) & 1);
            for (int g = max(0, gk - kSKStages); g < gk; g++)
                mbar_wait_asleep(&k_full[g % kSKStages], (g / kSKStages) & 1);
            for (; gc < gr; gc++)
                mbar_wait_asleep(&raw[gc & 1], (gc >> 1) & 1);
            for (int g = max(0, gv - kSRStages); g < gv; g++)
                mbar_wait_asleep(&r_full[g % kSRStages], (g / kSRStages) & 1);
        }
        __syncwarp();
    } else if (warp == kTcMmaWarp || warp == kTcMmaWarp + 1) {
        // ----------------------------------------------------------------- MMA
        // One warp per query tile t.  Per key tile j: P.V_t(j), then, once it has
        // read P_t(j), S_t(j + 1) into the same buffer.  The two warps take turns (a
        // lock in shared memory) with such a pair: a tile's MMAs then run back to
        // back while the other tile's softmax works.  Without it both tiles' MMAs
        // share the pipe, both softmax groups get their scores at the same time, and
        // the pipe idles while both work (a long chunk 747 -> 816 us).
        // A K, V or Q stage is released by one arrival per query tile: V by this warp,
        // which waits for its P.V, K and Q by the softmax group as it finds S_t(j), or
        // by this warp, for a stage its tile does not read, once that stage's tile has
        // landed (so that the arrival counts towards that tile's phase).  Plain
        // arrivals: each further commit costs the issuing thread about 100 cycles.
        const int t = warp - kTcMmaWarp;
        bool ok = true;
        const uint32_t qt = smem_u32(sQ) + (uint32_t)t * kQTile;
        const uint32_t idS = tc::idesc_e4m3(kTcRows, kSKeys);
        const uint32_t idO = tc::idesc_f16(kTcRows, D, true);
        const uint32_t dS = tmem + 256u + 128u * (uint32_t)t, dO = tmem + 128u * (uint32_t)t;
        // K rows of D codes, swizzled at their width
        const auto k_desc = [](uint32_t at) {
            return D == 128 ? tc::smem_desc(at, 16, 1024) : tc::smem_desc_64b(at, 16, 512);
        };
        if (tc::elect_one()) {
            int g0 = 0;    // K/V tiles of the previous items
            int gq = 0;    // S/P tiles of this query tile so far
            int used = 0;  // items in which this query tile had work
            for (int n = 0; ok; n++) {
                if (!(ok = mbar_wait_asleep(&item_ready[n & 1], (n >> 1) & 1)))
                    break;
                const PrefillItem it = items[n & 1].f;
                if (it.b < 0)
                    break;
                const int nk = it.nkt[t];
                const int nkt = max(it.nkt[0], it.nkt[1]);
                if (nk > 0 && !(ok = mbar_wait_asleep(&q_conv[t], used & 1)))
                    break;
                tc::fence_after();
                for (int w = 0; nk == 0 && w < 4; w++)  // this tile reads no Q this item
                    mbar_arrive(&q_empty[t]);
                // S_t(j), its K tile landed and S_t's buffer free
                auto scores = [&](int j) {
                    const int s = (g0 + j) % kSKStages;
                    tc::fence_after();
                    const uint32_t ka = smem_u32(sK + (size_t)s * kTile);
                    // Q = high + low part, both in one accumulator: the second part lies
                    // behind the first, D = 128 in the other half, D = 64 in the same rows
#pragma unroll
                    for (int kq = 0; kq < 2 * (D / 32); kq++) {
                        const uint32_t step = (uint32_t)(kq % (D / 32)) * 32;
                        const uint32_t offq = kq < D / 32 ? step : step + (D == 128 ? kQHalf : 64u);
                        tc::mma_ss_f8(dS, tc::smem_desc(qt + offq, 16, 1024), k_desc(ka + step), idS, kq > 0);
                    }
                    tc::commit(smem_u32(&s_full[t]));
                };
                auto landed = [&](int j) {
                    return mbar_wait_asleep(&k_full[(g0 + j) % kSKStages], ((g0 + j) / kSKStages) & 1);
                };
                if (nk > 0) {
                    // the buffer is free: this warp saw the previous item's last P.V complete
                    if (!(ok = landed(0)) || !(ok = turn.take()))
                        break;
                    scores(0);
                    turn.pass();
                }
                for (int j = 0; j < nk; j++) {
                    // P.V_t(j) once P_t(j) is written and V tile j converted; and, so that
                    // nothing is waited for that the other warp may owe while the turn is
                    // held, K tile j + 1 landed
                    const int s = (g0 + j) % kSVStages;
                    if (!(ok = mbar_wait_asleep(&v_conv[s], ((g0 + j) / kSVStages) & 1)))
                        break;
                    // the item's first P.V overwrites O: the tile's previous epilogue
                    // must have read it out
                    if (j == 0 && used >= 1 && !(ok = mbar_wait_asleep(&o_free[t], (used - 1) & 1)))
                        break;
                    if (j + 1 < nk && !(ok = landed(j + 1)))
                        break;
                    // keys 64 .. 127 first: their P is written first, and their MMAs run
                    // while the softmax is at the other half
                    const uint32_t va = smem_u32(sV + (size_t)s * kVTile);
                    auto pv = [&](int half, bool add) {
                        tc::fence_after();
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int kk = 4 * half + i;
                            tc::mma_ts(dO, dS + 96u * half + 8u * i,
                                       tc::smem_desc(va + 2048u * kk, kVHalf, 1024), idO,
                                       (add || i > 0) ? 1u : 0u);
                        }
                    };
                    if (!(ok = mbar_wait_asleep(&pv_ready[2 + t], gq & 1)) || !(ok = turn.take()))
                        break;
                    pv(1, j > 0);
                    turn.pass();
                    if (!(ok = mbar_wait_asleep(&pv_ready[t], gq & 1)) || !(ok = turn.take()))
                        break;
                    pv(0, true);
                    tc::commit(smem_u32(&pv_done[t]));
                    // S_t(j + 1) overwrites P_t(j)
                    ok = mbar_wait_asleep(&pv_done[t], gq & 1);
                    gq++;
                    if (ok) {
                        mbar_arrive(&v_empty[s]);
                        if (j + 1 < nk)
                            scores(j + 1);
                    }
                    turn.pass();
                    if (!ok)
                        break;
                }
                // K and V tiles that this query tile does not read
                for (int j = nk; ok && j < nkt; j++) {
                    const int s = (g0 + j) % kSVStages;
                    if (!(ok = landed(j)))
                        break;
                    for (int w = 0; w < 4; w++)  // for its softmax warps
                        mbar_arrive(&k_empty[(g0 + j) % kSKStages]);
                    if (!(ok = mbar_wait_asleep(&v_conv[s], ((g0 + j) / kSVStages) & 1)))
                        break;
                    mbar_arrive(&v_empty[s]);
                }
                if (!ok)
                    break;
                g0 += nkt;
                used += nk > 0 ? 1 : 0;
                mbar_arrive(&item_free[n & 1]);
            }
            if (!ok)
                flag_error(p.err_flag, 0x8 /* PKV_FLAG_TIMEOUT */);
            tc::commit(smem_u32(mma_done));  // every MMA completes before TMEM is released
        }
        __syncwarp();
        mbar_wait_asleep(mma_done, 0);
        __syncwarp();
    } else {
        // ------------------------------------------------------------- softmax
        const int tq = warp >> 2;            // query tile of this group (A = 0, B = 1)
        const int r = threadIdx.x & 127;     // row = TMEM lane
        const uint32_t tl = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tO = tmem + 128u * tq + tl, tS = tmem + 256u + 128u * tq + tl;
        bool ok = true;
        int g0 = 0, gq = 0;
        int used = 0;  // items in which this query tile had work
        // Conversion of this group's half of a V tile: a thread turns 16 codes of rows
        // conv_row + kConvStep u.  Eight lanes take four pieces each of two rows, for
        // D = 128 of different halves: that way their reads and either of their writes
        // touch all banks.
        constexpr int kConvPieces = 64 * (D / 16) / 128, kConvStep = 64 / kConvPieces;
        const int conv_row = 64 * tq + (D == 128 ? 2 * (r >> 4) + ((r >> 2) & 1) : r >> 2);
        const int conv_col = D == 128 ? (r & 3) + 4 * (((r >> 2) ^ (r >> 3)) & 1) : r & 3;
        const int conv_from = conv_row * D + 16 * (D == 128 ? conv_col ^ (conv_row & 7)
                                                            : conv_col ^ ((conv_row >> 1) & 3));
        const int conv_line = (conv_col >> 2) * (int)kVHalf + conv_row * 128;
        const int conv_to0 = conv_line + 16 * ((2 * (conv_col & 3)) ^ (conv_row & 7));
        const int conv_to1 = conv_line + 16 * ((2 * (conv_col & 3) + 1) ^ (conv_row & 7));
        for (int n = 0; ok; n++) {
            ok = __all_sync(FULL, mbar_wait_asleep(&item_ready[n & 1], (n >> 1) & 1));
            if (!ok)
                break;
            const WideItem item = items[n & 1];
            const PrefillItem &it = item.f;
            if (it.b < 0)
                break;
            const int nkt = it.nkt[tq], all = max(it.nkt[0], it.nkt[1]);
            const int j0 = SPLIT ? item.j0 : 0;
            const int tok = it.tok0 + tq * TPC + r / G, g = r % G;
            const bool valid = tok < it.q_len;
            const int pos = (it.k_len - it.q_len) + tok;
            const int k_len = it.k_len;
            float m = -INFINITY, l = 0.f;
            // of the next key tile's codes, and of this row's O
            float unit = 1.f, o_unit = 1.f;
            uint32_t boxes = 0;  // `read` of the next key tile
            // Key tile j's scales, and this group's half (64 keys) of its V: codes -> f16 in
            // the other buffer, times their box's factor, rows past k_len or of boxes that
            // are not read zeroed (their weight is 0, and 0 * NaN would be NaN).  Both groups
            // take part in every tile of the item, in order.
            auto convert_v = [&](int j) -> bool {
                const int gv = g0 + j, s = gv % kSRStages, b = gv % kSVStages, kb = (j0 + j) * kSKeys;
                if (!__all_sync(FULL, mbar_wait_asleep(&r_full[s], (gv / kSRStages) & 1)))
                    return false;
                const uint8_t *vr = sR + (size_t)s * kTile + conv_from;
                uint4 w[kConvPieces];
#pragma unroll
                for (int u = 0; u < kConvPieces; u++)
                    w[u] = *reinterpret_cast<const uint4 *>(vr + u * kConvStep * D);
                const TileScales &ts = scales[gv % kSScales];
                uint32_t f[kConvPieces];
#pragma unroll
                for (int u = 0; u < kConvPieces; u++)
                    f[u] = ts.v[(conv_row + u * kConvStep) / kBox];
                const int2 rest = *reinterpret_cast<const int2 *>(&ts.read);
                boxes = (uint32_t)rest.x;
                unit = __int_as_float(rest.y);
                uint8_t *vt = sV + (size_t)b * kVTile;
                const bool clear = boxes != 0xffu || kb + kSKeys > k_len;
#pragma unroll
                for (int u = 0; u < kConvPieces; u++) {
                    uint4 x = e4m3x8_to_f16(w[u].x, w[u].y, f[u]), y = e4m3x8_to_f16(w[u].z, w[u].w, f[u]);
                    if (clear) {
                        const int row = conv_row + u * kConvStep;
                        if (kb + row >= k_len || !((boxes >> (row / kBox)) & 1u))
                            x = y = make_uint4(0u, 0u, 0u, 0u);
                    }
                    *reinterpret_cast<uint4 *>(vt + conv_to0 + u * kConvStep * 128) = x;
                    *reinterpret_cast<uint4 *>(vt + conv_to1 + u * kConvStep * 128) = y;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&r_empty[s]);
                    mbar_arrive(&v_conv[b]);
                }
                return true;
            };
            // This row of Q as two E4M3 parts, q = sq (high + low), in its own place.  With
            // sq = 2^(E - 7) for max|q| in [2^E, 2^(E + 1)) the sum is exact for every
            // element of magnitude >= max|q| 2^-9 and within max|q| 2^-17 for the rest
            // (E4M3's least step is 2^-9).  A negative softmax scale negates the parts; an
            // infinite element makes the row NaN.
            float sl = 0.f;  // score -> log2 units, but for K's scale
            if (nkt > 0) {
                if (!(ok = __all_sync(FULL, mbar_wait_asleep(&q_full[tq], used & 1))))
                    break;
                used++;
                uint8_t *qr = sQ + (size_t)tq * kQTile + r * 128;
                const auto at = [&](int i) {  // sixteen bytes of the row
                    return reinterpret_cast<uint4 *>(qr + (i >> 3) * kQHalf + (((i & 7) ^ (r & 7)) << 4));
                };
                uint32_t top = 0;  // two bf16 magnitudes
#pragma unroll 4
                for (int i = 0; i < D / 8; i++) {
                    const uint4 w = *at(i);
                    top = bf16x2_absmax(top, bf16x2_absmax(bf16x2_absmax(w.x, w.y), bf16x2_absmax(w.z, w.w)));
                }
                top &= 0x7fff7fffu;
                top = max(top & 0xffffu, top >> 16);
                const int ebits = min(max((int)(top >> 7), 8), 254);
                // (not so small that its product with a K scale is 0, which times a masked score,
                // -inf, would be NaN, or that log2 g over it is infinite: no score that small moves
                // a weight)
                sl = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(ebits - 7) << 23), 1e-24f);
                if (top == 0x7f80u)
                    sl = NAN;
                float inv = __uint_as_float((uint32_t)(261 - ebits) << 23);
                if (p.neg_scale)
                    inv = -inv;
                const float2 inv2 = make_float2(inv, inv);
                // The high parts fill the row's first half, behind what is read; the low parts
                // its second, once all is read: until then they lie in the score columns.  A
                // loop, for its instructions' sake.
#pragma unroll 1
                for (int i = 0; i < D / 16; i++) {  // sixteen elements
                    const uint4 w0 = *at(2 * i), w1 = *at(2 * i + 1);
                    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        const float2 a0 = fmul2(bf16x2_to_float2(w[2 * c]), inv2),
                                     a1 = fmul2(bf16x2_to_float2(w[2 * c + 1]), inv2);
                        // (in f16 both are exact, but for what lies below 2^-14)
                        const uint32_t x0 = pack_f16x2(a0.x, a0.y), x1 = pack_f16x2(a1.x, a1.y);
                        const uint32_t h0 = f16x2_to_e4m3x2(x0), h1 = f16x2_to_e4m3x2(x1);
                        hi[c] = h0 | (h1 << 16);
                        lo[c] = f16x2_to_e4m3x2(f16x2_sub(x0, e4m3x2_to_f16x2(h0))) |
                                (f16x2_to_e4m3x2(f16x2_sub(x1, e4m3x2_to_f16x2(h1))) << 16);
                    }
                    *at(i) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    tc::st4(tS + 4 * i, lo);
                }
                tc::wait_st();
                uint32_t lo[D / 4];
                if constexpr (D == 128)
                    tc::ld32(tS, lo);
                else
                    tc::ld16(tS, lo);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < D / 16; i++)
                    *at(D / 16 + i) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                tc::fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&q_conv[tq]);
            }
            if (!(ok = convert_v(0)))
                break;
            for (int j = 0; j < nkt; j++) {
                const int gt = gq + j;
                ok = __all_sync(FULL, mbar_wait_asleep(&s_full[tq], gt & 1));
                if (!ok)
                    break;
                tc::fence_after();
                // S_t(j) has completed: its K tile, and after the item's last one its
                // Q, is read
                if (lane == 0) {
                    mbar_arrive(&k_empty[(g0 + j) % kSKStages]);
                    if (j == nkt - 1)
                        mbar_arrive(&q_empty[tq]);
                }
                const int key_base = (j0 + j) * kSKeys;
                const TileScales &ts = scales[(g0 + j) % kSScales];
                // Masked keys, past their row's position (the diagonal tiles) or in a box that
                // is not read: -inf into the scores, so that what follows knows of none.  Most
                // tiles have none in the whole warp; of its own and short, because the
                // instructions of the rest barely fit the caches.
                if (__any_sync(FULL, boxes != 0xffu || key_base + kSKeys - 1 > pos)) {
                    const int lim = pos - key_base;  // keys i > lim are in the future
#pragma unroll 1
                    for (int b = 0; b < kBoxes; b++) {
                        const int last = (boxes >> b) & 1u ? lim - kBox * b : -1;
                        if (__all_sync(FULL, last >= kBox - 1))
                            continue;
                        uint32_t r[16];
                        tc::ld16(tS + kBox * b, r);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < kBox; i++)
                            r[i] = i > last ? __float_as_uint(-INFINITY) : r[i];
                        tc::st16(tS + kBox * b, r);
                    }
                    tc::wait_st();
                    if (__builtin_expect(boxes >> kBoxes, 0)) {
                        const RowState now = odd_scales<D>(tS, tO, ts, boxes, lim, sl, {m, l, unit, o_unit}, j > 0);
                        m = now.m;
                        l = now.l;
                        unit = now.unit;
                        o_unit = now.o_unit;
                    }
                }
                // K's scales of the tile's boxes join the row's
                const float *ks = ts.k;
                float x[64];
                auto load = [&](int half) {
                    uint32_t a[32], b[32];
                    tc::ld32(tS + 64 * half, a);
                    tc::ld32(tS + 64 * half + 32, b);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        x[i] = __uint_as_float(a[i]);
                        x[32 + i] = __uint_as_float(b[i]);
                    }
                };
                auto top = [&](int half, float t) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(ks + 4 * half);
#pragma unroll
                    for (int b = 0; b < 4; b++) {
                        const float *y = x + kBox * b;
                        const float u = max3(max3(y[0], y[1], y[2]), max3(y[3], y[4], y[5]), max3(y[6], y[7], y[8]));
                        const float v = max3(max3(y[9], y[10], y[11]), max3(y[12], y[13], y[14]), y[15]);
                        t = fmaxf(t, fmaxf(u, v) * (b == 0 ? k4.x : b == 1 ? k4.y : b == 2 ? k4.z : k4.w));
                    }
                    return t;
                };
                load(0);
                float mraw = top(0, -INFINITY);
                load(1);
                mraw = top(1, mraw);
                const float mx = mraw * sl;
                if (__any_sync(FULL, mx > m + kLazy || unit != o_unit)) {
                    const float mn = fmaxf(m, mx);
                    const float alpha = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
                    const float o_alpha = alpha * exp2_ratio(o_unit, unit);
                    o_unit = unit;
                    if (j > 0)
                        rescale_o<D>(tO, o_alpha);
                    l *= alpha;
                    m = mn;
                }
                const float nmu = m == -INFINITY ? 0.f : -m;
                const float2 nm2 = make_float2(nmu, nmu);
                float2 ls0 = make_float2(0.f, 0.f), ls1 = ls0;
                auto exponentiate = [&](int half, uint32_t to) {
                    uint32_t pk[32];
                    const float4 k4 = *reinterpret_cast<const float4 *>(ks + 4 * half);
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const float c = sl * (i < 8 ? k4.x : i < 16 ? k4.y : i < 24 ? k4.z : k4.w);
                        const float2 a = ffma2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(c, c), nm2);
                        const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                        if (i & 1)
                            ls1 = fadd2(ls1, e);
                        else
                            ls0 = fadd2(ls0, e);
                        pk[i] = pack_f16x2(e.x, e.y);
                    }
                    tc::st32(to, pk);
                };
                auto hand_over = [&](int half) {
                    tc::wait_st();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&pv_ready[2 * half + tq]);
                };
                // Keys 64..127 first, over score columns read above; then keys 0..63 again.
                // One copy of the instructions, but where there are few items of long
                // contexts (SPLIT), which run a tile's 1% faster in two and have the fewest
                // other instructions between: 8 x 2048 on nothing 144 us (154 in two copies),
                // on 2048 341 (353), 32 x 512 on 512 244 (266), on 14336 1481 (1470); SPLIT,
                // 2048 on 28672 780 (748).
#pragma unroll(SPLIT ? 2 : 1)
                for (int h = 1; h >= 0; h--) {
                    if (h == 0)
                        load(0);
                    exponentiate(h, tS + 96 * h);
                    hand_over(h);
                }
                l += (ls0.x + ls0.y) + (ls1.x + ls1.y);
                // off the chain: V tile j + 1 while P.V_t(j) and S_t(j + 1) run
                if (j + 1 < all && !(ok = convert_v(j + 1)))
                    break;
            }
            if (!ok)
                break;
            // V tiles that only the other query tile reads
            for (int jv = max(nkt, 1) + (nkt > 0 ? 1 : 0); ok && jv < all; jv++) {
                ok = convert_v(jv);
            }
            if (!ok)
                break;
            // a split that only the other query tile has keys in
            const bool piece = SPLIT && item.split >= 0;
            if (piece && nkt == 0 && valid)
                p.part_lse[(size_t)item.split * p.Tq * p.Hq +
                           ((size_t)it.kvh * p.Tq + it.cq0 + tok) * G + g] = -INFINITY;
            if (nkt > 0) {
                const int gl = gq + nkt - 1;
                ok = __all_sync(FULL, mbar_wait_asleep(&pv_done[tq], gl & 1));
                if (!ok)
                    break;
                tc::fence_after();
                const float inv = l > 0.f ? o_unit / l : 0.f;
                float any = 0.f;  // NaN if an element of the row is
                const auto pair = [](const uint32_t *o) {
                    return make_float2(__uint_as_float(o[0]), __uint_as_float(o[1]));
                };
                const size_t row = (size_t)it.cq0 + tok;
                const size_t lse_at = ((size_t)it.kvh * p.Tq + row) * G + g;
                if (piece) {
                    // this split's output in fp32, and its log-sum-exp (-inf: no key)
                    if (valid)
                        p.part_lse[(size_t)item.split * p.Tq * p.Hq + lse_at] =
                            l == 0.f ? -INFINITY : m + log2f(l);
                    float *dst = p.part_out + (((size_t)item.split * p.Tq + row) * p.Hq + it.kvh * G + g) * D;
                    const bool aligned32 = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; cc++) {
                        uint32_t ro[32];
                        tc::ld32(tO + 32 * cc, ro);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 y = fmul2(pair(ro + i), make_float2(inv, inv));
                            any = max3_nan(any, y.x, y.y);
                            ro[i] = __float_as_uint(y.x);
                            ro[i + 1] = __float_as_uint(y.y);
                        }
#pragma unroll
                        for (int i = 0; i < 32 && valid; i += 8)
                            store32(dst + 32 * cc + i, ro + i, aligned32);
                    }
                } else {
                    if (SPLIT && valid)
                        p.part_lse[lse_at] = INFINITY;  // nothing to join
                    // a row per thread in 32-byte pieces: whole sectors
                    uint16_t *dst = p.out + (row * p.Hq + it.kvh * G + g) * D;
                    const bool aligned32 = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; cc++) {
                        uint32_t ro[32], v[16];
                        tc::ld32(tO + 32 * cc, ro);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            const float2 y = fmul2(pair(ro + 2 * i), make_float2(inv, inv));
                            any = max3_nan(any, y.x, y.y);
                            v[i] = pack_bf16x2(y.x, y.y);
                        }
                        if (valid) {
                            store32(dst + 32 * cc, v, aligned32);
                            store32(dst + 32 * cc + 16, v + 8, aligned32);
                        }
                    }
                }
                // A NaN that is not the scores': one in V, which a weight of 0 (a row that does
                // not see its token) makes one too.  The item once more, from codes without
                // them, and then NaN where a row sees one.
                if (any != any && l == l && valid && !item.clean)
                    again[n & 1] = 1;
                if (__builtin_expect(item.clean, 0) && valid) {
                    const size_t at = (row * p.Hq + it.kvh * G + g) * D;
                    if (piece)
                        write_nans<D>(p.part_out + (size_t)item.split * p.Tq * p.Hq * D + at, NAN,
                                      nan_from + (n & 1) * D, pos);
                    else
                        write_nans<D>(p.out + at, (uint16_t)0x7fff, nan_from + (n & 1) * D, pos);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&o_free[tq]);  // the tile's next first P.V may overwrite O
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&item_free[n & 1]);
            g0 += all;
            gq += nkt;
        }
        if (!ok && lane == 0)
            flag_error(p.err_flag, 0x8 /* PKV_FLAG_TIMEOUT */);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kTcMmaWarp) {
        tc::fence_after();
        tc::dealloc(tmem, kTcCols);
    }
}

template <int D>
inline cudaError_t launch_prefill_scaled_d(int G, const CUtensorMap *tmq, const CUtensorMap *tmk,
                                         const CUtensorMap *tmv, const PrefillParams &p, dim3 grid,
                                         size_t smem, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (G) {
    case 1:
        return p.splits > 1 ? cudaLaunchKernelEx(&cfg, paged_prefill_scaled_kernel<D, 1, true>, *tmq, *tmk, *tmv, p)
                            : cudaLaunchKernelEx(&cfg, paged_prefill_scaled_kernel<D, 1, false>, *tmq, *tmk, *tmv, p);
    case 2:
        return p.splits > 1 ? cudaLaunchKernelEx(&cfg, paged_prefill_scaled_kernel<D, 2, true>, *tmq, *tmk, *tmv, p)
                            : cudaLaunchKernelEx(&cfg, paged_prefill_scaled_kernel<D, 2, false>, *tmq, *tmk, *tmv, p);
    case 4:
        return p.splits > 1 ? cudaLaunchKernelEx(&cfg, paged_prefill_scaled_kernel<D, 4, true>, *tmq, *tmk, *tmv, p)
                            : cudaLaunchKernelEx(&cfg, paged_prefill_scaled_kernel<D, 4, false>, *tmq, *tmk, *tmv, p);
    case 8:
        return p.splits > 1 ? cudaLaunchKernelEx(&cfg, paged_prefill_scaled_kernel<D, 8, true>, *tmq, *tmk, *tmv, p)
                            : cudaLaunchKernelEx(&cfg, paged_prefill_scaled_kernel<D, 8, false>, *tmq, *tmk, *tmv, p);
    default: return cudaErrorInvalidValue;
    }
}

template <int D> inline const void *prefill_scaled_kernel_d(int G, bool split)
{
    switch (G) {
    case 1:
        return split ? reinterpret_cast<const void *>(&paged_prefill_scaled_kernel<D, 1, true>)
                     : reinterpret_cast<const void *>(&paged_prefill_scaled_kernel<D, 1, false>);
    case 2:
        return split ? reinterpret_cast<const void *>(&paged_prefill_scaled_kernel<D, 2, true>)
                     : reinterpret_cast<const void *>(&paged_prefill_scaled_kernel<D, 2, false>);
    case 4:
        return split ? reinterpret_cast<const void *>(&paged_prefill_scaled_kernel<D, 4, true>)
                     : reinterpret_cast<const void *>(&paged_prefill_scaled_kernel<D, 4, false>);
    case 8:
        return split ? reinterpret_cast<const void *>(&paged_prefill_scaled_kernel<D, 8, true>)
                     : reinterpret_cast<const void *>(&paged_prefill_scaled_kernel<D, 8, false>);
    default: return nullptr;
    }
}

} // namespace pkv
