// store_kvcache_scaled: new K/V rows into an E4M3 cache whose scales lie per block and
// KV head (fp32 [NB, Hkv], for K and for V).
//
// Mathematics.  For a block, a KV head and K or V alike, with a = the largest finite
// magnitude that the call stores there, the scale that holds them is 2^e with the
// least e in [-40, 40] for which a <= 448 * 2^e.  E4M3 being a floating format, a power
// of two costs no precision beside a / 448, and a scale that grows by a power of two
// recodes old rows exactly (but for codes that become subnormal), however often.
//   * A call that stores a block's first token (offset 0) begins it: the scale is 2^e,
//     whatever stood there.  So does one that finds no positive finite scale.
//   * Else s' = max(s, 2^e); where s' > s, every row of the block and head is recoded by
//     s / s' before the call's rows are written over it.
// Codes: e4m3(x * (1 / s')), exact products where s' is a power of two.
//
// How.  A block's tokens follow each other in slot_mapping (a run).  One CTA takes the
// runs that start in a window of T tokens, for one KV head and K or V: it keeps a
// batch of the rows that it reads in registers (those before the last batch are read
// again, from L2), takes each run's maximum in shared memory, and writes.  So the
// scale needs no second kernel and no workspace.
//
// Measured (8 KV heads, D = 128): 16384 tokens, 101 MB, in blocks of 256 or of 16 21 to 25 us
// over and over, 0.59 to 0.71 of the rate of a plain copy (L2 holds part of them), 27 us, 0.55,
// with caches flushed; a step of 256 sequences 2.6 us behind another one.
// Bound by a CTA's chain (slots, rows, maximum, scale, rows again) at four CTAs an SM,
// whose issue slots are 60% used.  Not kept: 16-byte loads, twice the lanes per row
// (28 us), twice the rows in registers and half the CTAs (28), windows of 64 tokens (26),
// 512 threads (25), K and V by one CTA (4096 tokens 15.6 for 10.8).
#include "pkv_kernels.h"
#include "pkv_ptx.cuh"
#include "pkv_quant.cuh"
#include "pkv_scaled.h"

namespace pkv {

constexpr int kSsThreads = 256;
constexpr int kScaleLow = -40, kScaleHigh = 40;

// Sixteen bf16 values.
struct Row16 {
    uint32_t w[8];
};

__device__ __forceinline__ Row16 load16(const uint8_t *p, bool aligned32)
{
    Row16 r;
    if (!aligned32) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p)), b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
        return r;
    }
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]),
                   "=r"(r.w[6]), "=r"(r.w[7])
                 : "l"(p));
    return r;
}

// Bits of the largest finite magnitude (0 where there is none).
__device__ __forceinline__ uint32_t finite_max16(const Row16 &r)
{
    uint32_t m = bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(r.w[0], r.w[1]), bf16x2_absmax(r.w[2], r.w[3])),
                               bf16x2_absmax(bf16x2_absmax(r.w[4], r.w[5]), bf16x2_absmax(r.w[6], r.w[7]))) &
                 0x7fff7fffu;
    m = max(m & 0xffffu, m >> 16);
    if (m >= 0x7f80u) {  // infinities, or nothing but NaN in a place of all eight
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t lo = r.w[i] & 0x7fffu, hi = (r.w[i] >> 16) & 0x7fffu;
            m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
    }
    return m;
}

// The least power of two in range that holds a magnitude (bf16 bits).
__device__ __forceinline__ float scale_for(uint32_t m)
{
    // m = 1.f * 2^(E - 127), 448 = 1.75 * 2^8
    int e = (int)(m >> 7) - 127 - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0);
    e = min(max(e, kScaleLow), kScaleHigh);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// T: tokens per window.  SEEN: tokens from the window's first on whose slots are looked
// at at once.  HOLD: row loads a thread has in flight and keeps.
template <int D, int T, int SEEN, int HOLD>
__global__ void __launch_bounds__(kSsThreads) store_scaled_kernel(const StoreScaledParams p)
{
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int LPR = D / 16;             // lanes per row (32-byte loads)
    constexpr int RPP = kSsThreads / LPR;   // rows per pass
    constexpr int BATCH = HOLD * RPP;       // rows kept
    constexpr int PER = SEEN / kSsThreads;  // slots per thread
    constexpr int WARPS = kSsThreads / 32;
    static_assert(SEEN % kSsThreads == 0 && T <= kSsThreads && T < SEEN && T % 16 == 0, "window");
    __shared__ int s_slot[SEEN + 1], s_of[SEEN + 1];  // slot and block of tokens w0 - 1, w0, ...; -1: none
    __shared__ short s_run[SEEN];           // run of each token, -1: none that starts here
    __shared__ uint32_t s_start[WARPS], s_goes[SEEN / 32];  // a bit per token
    __shared__ int s_blk[T];
    __shared__ uint32_t s_max[T], s_begun[T];
    __shared__ float s_inv[T], s_ratio[T];
    __shared__ int s_grown[T];
    __shared__ int s_n_grown;
    __shared__ long long s_end;

    grid_launch_dependents();
    // Earlier kernels may have written any of the inputs, and may still read the cache.
    // (With the inputs read ahead of this, a step behind another one 1.8 us, so 2.5.)
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // K and V, then heads, then windows: CTAs that run together read the same rows
    const int z = blockIdx.x & 1, h = (int)((blockIdx.x >> 1) % (uint32_t)p.Hkv);
    const long long w0 = (long long)((blockIdx.x >> 1) / (uint32_t)p.Hkv) * T;
    const uint32_t bs = (uint32_t)p.bs;

    // ---- the window's runs: a token starts one unless the token before it lies in its block
    const auto slot_at = [&](long long i) -> int {
        const long long s = i >= 0 && i < p.N ? __ldg(p.slots + i) : -1;
        if (s >= 0 && s < p.n_slots)
            return (int)s;
        if (s != -1 && h == 0 && z == 0)
            flag_error(p.err_flag, 0x1 /* PKV_FLAG_BAD_SLOT */);
        return -1;
    };
    const auto block_of = [&](int s) { return s >= 0 ? divide(s, p.block) : -1; };
    int slots[PER];
#pragma unroll
    for (int i = 0; i < PER; i++)
        slots[i] = slot_at(w0 + i * kSsThreads + tid);
    if (tid == 0) {
        s_of[0] = block_of(slot_at(w0 - 1));
        s_n_grown = 0;
    }
#pragma unroll
    for (int i = 0; i < PER; i++) {
        s_slot[1 + i * kSsThreads + tid] = slots[i];
        s_of[1 + i * kSsThreads + tid] = block_of(slots[i]);
    }
    if (tid < T)
        s_max[tid] = s_begun[tid] = 0;
    __syncthreads();
    const int slot = slots[0], blk = s_of[1 + tid];
    bool start = false;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int t = i * kSsThreads + tid;
        const bool follows = s_of[t + 1] >= 0 && s_of[t] == s_of[t + 1];
        if (i == 0)
            start = tid < T && slot >= 0 && !follows;
        const uint32_t goes = __ballot_sync(FULL, follows);
        if (lane == 0)
            s_goes[t >> 5] = goes;
    }
    const uint32_t starts = __ballot_sync(FULL, start);
    if (lane == 0)
        s_start[warp] = starts;
    __syncthreads();
    const uint32_t begin = lane < WARPS ? s_start[lane] : 0u;
    const uint32_t some = __ballot_sync(FULL, begin != 0u);
    if (some == 0u)
        return;
    const int n_runs = __reduce_add_sync(FULL, __popc(begin));
    const int before = __reduce_add_sync(FULL, lane < warp ? __popc(begin) : 0);
    const int at = __ffs(some) - 1;
    const int first = 32 * at + __ffs(__shfl_sync(FULL, begin, at)) - 1;
    // how far the last run goes on behind the window, of what is seen (a lane per word)
    static_assert(SEEN / 32 <= 32, "a lane per word");
    uint32_t stops = lane < SEEN / 32 ? ~s_goes[lane] : 0u;
    if (32 * lane < T)
        stops = T - 32 * lane >= 32 ? 0u : stops & (FULL << (T - 32 * lane));
    const uint32_t words = __ballot_sync(FULL, stops != 0u);
    const int word = words ? __ffs(words) - 1 : 0;
    const uint32_t stop = __shfl_sync(FULL, stops, word);
    const int end = words ? 32 * word + __ffs(stop) - 1 : SEEN;
    if (tid < T) {
        const int run = slot >= 0 ? before + __popc(starts & (FULL >> (31 - lane))) - 1 : -1;
        s_run[tid] = (short)run;
        if (start)
            s_blk[run] = blk;
        if (run >= 0 && (uint32_t)slot == (uint32_t)blk * bs)
            s_begun[run] = 1;
    }
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int t = i * kSsThreads + tid;
        if (t >= T) {
            s_run[t] = (short)(n_runs - 1);
            if (t < end && (uint32_t)slots[i] == (uint32_t)s_of[t + 1] * bs)
                s_begun[n_runs - 1] = 1;
        }
    }
    if (tid == 0)
        s_end = min(w0 + end, p.N);
    if (end == SEEN) {  // and beyond
        __syncthreads();
        const int last = s_of[SEEN];
        for (long long i = w0 + SEEN + tid;; i += kSsThreads) {
            const int s = slot_at(i);
            const bool mine = block_of(s) == last;
            if (mine && (uint32_t)s == (uint32_t)last * bs)
                s_begun[n_runs - 1] = 1;
            const int other = __syncthreads_or(!mine);
            if (other) {
                if (tid == 0)
                    s_end = p.N;
                __syncthreads();
                if (!mine && i < p.N)
                    atomicMin(&s_end, i);
                break;
            }
        }
    }
    __syncthreads();

    // ---- each run's largest magnitude; row i is token w0 + first + i
    const long long row0 = w0 + first;
    const int rows = (int)(s_end - row0);
    const int sub = tid / LPR, part = tid % LPR;
    const auto run_of = [&](int i) { return first + i < SEEN ? (int)s_run[first + i] : n_runs - 1; };
    const size_t stride = (size_t)p.Hkv * D * 2;
    const uint8_t *src = (z ? p.x[1] : p.x[0]) + row0 * stride + (size_t)h * D * 2 + part * 32;
    const bool aligned32 = (reinterpret_cast<uintptr_t>(src) & 31u) == 0;  // of all or none
    Row16 held[HOLD];
    const auto load = [&](int b0) {  // (behind the last row: that one again)
#pragma unroll
        for (int u = 0; u < HOLD; u++) {
            held[u] = load16(src + (size_t)min(b0 + u * RPP + sub, rows - 1) * stride, aligned32);
        }
    };
    load(0);
    float *scale_at = nullptr;
    float had = 0.f;
    if (tid < n_runs) {
        scale_at = (z ? p.scales[1] : p.scales[0]) + (size_t)s_blk[tid] * p.Hkv + h;
        had = ld_gpu(scale_at);
    }
    // a thread's rows ascend, and so do their runs: it gathers while the run stays
    uint32_t top = 0;
    int of = -1;
    const auto flush = [&]() {  // by all lanes of a warp
        const int lead = __shfl_sync(FULL, of, 0);
        if (__all_sync(FULL, of == lead)) {
            const uint32_t m = __reduce_max_sync(FULL, top);
            if (lane == 0 && of >= 0)
                atomicMax(&s_max[of], m);
        } else if (of >= 0) {
            atomicMax(&s_max[of], top);
        }
    };
    int b0 = 0;
    for (;;) {
#pragma unroll
        for (int u = 0; u < HOLD; u++) {
            const int i = b0 + u * RPP;
            if (i >= rows)
                break;
            const int run = run_of(min(i + sub, rows - 1));
            if (__any_sync(FULL, run != of)) {
                flush();
                top = 0;
                of = run;
            }
            top = max(top, finite_max16(held[u]));
        }
        if (b0 + BATCH >= rows)
            break;
        b0 += BATCH;
        load(b0);
    }
    flush();
    __syncthreads();

    // ---- the scales
    if (tid < n_runs) {
        const float want = scale_for(s_max[tid]);
        const bool keep = !s_begun[tid] && had > 0.f && had < INFINITY;
        const float now = keep ? fmaxf(had, want) : want;
        s_inv[tid] = __frcp_rn(now);
        if (!keep || now != had)
            *scale_at = now;
        if (keep && now != had) {
            s_ratio[tid] = __fdiv_rn(had, now);
            s_grown[atomicAdd(&s_n_grown, 1)] = tid;
        }
    }
    __syncthreads();

    // ---- what grown blocks held before
    uint8_t *cache = z ? p.cache[1] : p.cache[0];
    const int n_grown = s_n_grown;
    if (n_grown > 0) {
        constexpr int CPR = D / 16;  // 16-byte pieces of a row of codes
        for (int g = 0; g < n_grown; g++) {
            const int run = s_grown[g];
            const float ratio = s_ratio[run];
            uint8_t *base = cache + ((size_t)s_blk[run] * bs * p.Hkv + h) * D;
            for (size_t c = tid; c < (size_t)bs * CPR; c += kSsThreads) {
                uint4 *w = reinterpret_cast<uint4 *>(base + c / CPR * p.Hkv * D + c % CPR * 16);
                const uint4 a = *w;
                *w = make_uint4(recode4(a.x, ratio), recode4(a.y, ratio), recode4(a.z, ratio),
                                recode4(a.w, ratio));
            }
        }
        __syncthreads();  // before rows of the same blocks are written over it
    }

    // ---- the rows, the batch that is held first
    cache += (size_t)h * D + part * 16;
    const size_t token = (size_t)p.Hkv * D;
    for (;;) {
#pragma unroll
        for (int u = 0; u < HOLD; u++) {
            const int i = b0 + u * RPP + sub;
            const int run = i < rows ? run_of(i) : -1;
            if (run >= 0) {
                const int s = first + i < SEEN ? s_slot[1 + first + i] : (int)__ldg(p.slots + row0 + i);
                const uint32_t *w = held[u].w;
                const float inv = s_inv[run];
                *reinterpret_cast<uint4 *>(cache + (size_t)(uint32_t)s * token) =
                    make_uint4(quantize4(w[0], w[1], inv), quantize4(w[2], w[3], inv), quantize4(w[4], w[5], inv),
                               quantize4(w[6], w[7], inv));
            }
        }
        if (b0 == 0)
            break;
        b0 -= BATCH;
        load(b0);
    }
}

template <int D> static cudaError_t launch(const StoreScaledParams &p, cudaStream_t stream)
{
    // Few rows of a head (decode steps, short chunks): small windows, so that more CTAs
    // share them.  More: windows of 128, whose look at the slots costs less per token.  What
    // decides is the number of CTAs, N * Hkv.  us in windows of 16 and of 128, one token in
    // each of N blocks, prompts of 200 tokens and of whole blocks in blocks of 16:
    //   N * Hkv = 2048   2.7-3.5 / 3.8   2.8-3.7 / 4.6   2.7-3.9 / 3.9
    //             4096   3.9 / 4.0       4.1 / 4.8       4.7-5.0 / 4.1
    //             8192   5.8 / 5.2       5.7 / 6.1       5.9 / 5.1
    //            16384   8.8 / 6.3       9.0 / 7.5       9.2 / 6.4
    // with 1, 2, 4 and 8 heads alike.  Prompts in large blocks have a CTA take a whole block
    // in either, and many that find nothing: 1024 tokens of 1 head in blocks of 256 6.5 / 5.2,
    // 4096 7.5 / 5.6; 512 of 8 heads 7.1 / 5.3.  So with blocks of more than 32 tokens, small
    // windows up to 512 tokens only, which are rather a step's (512 sequences of 1 head
    // 2.6 / 3.7, of 8 heads 3.9 / 4.0).
    // Where those of 128 are more than a round of CTAs (608), 256, in windows of 128 and of
    // 256: a chunk of 4096 in blocks of 16 8.4 / 10.8, of 6144 11.8 / 11.8, of 8192 14.0 / 13.4,
    // 16k tokens of ragged prompts 23.6 / 21.2, 32768 in blocks of 256 41.0 / 40.2 (16384 that
    // begin inside theirs 20.9 / 21.2); 32768 of 1 head 7.3 / 10.2, of 2 heads 12.1 / 12.0.
    const long long rows = p.N * p.Hkv;
    const bool few = rows <= 4096 && (p.N <= 512 || p.bs <= 32), many = !few && rows > 40960;
    const int T = few ? 16 : many ? 256 : 128;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((p.N + T - 1) / T * p.Hkv * 2));
    cfg.blockDim = dim3(kSsThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return few    ? cudaLaunchKernelEx(&cfg, store_scaled_kernel<D, 16, 256, 1>, p)
           : many ? cudaLaunchKernelEx(&cfg, store_scaled_kernel<D, 256, 512, D / 32>, p)
                  : cudaLaunchKernelEx(&cfg, store_scaled_kernel<D, 128, 512, D / 32>, p);
}

cudaError_t launch_store_scaled(int D, const StoreScaledParams &p, cudaStream_t stream)
{
    return D == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

} // namespace pkv
