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
// runs that start in a window of T tokens, for one KV head and K or V: it keeps the
// rows that it reads (256 of them at most; later ones of a run are read again, from
// L2) in registers, takes each run's maximum in shared memory, and writes.  So every
// row is read once and written once, and the scale needs no second kernel and no
// workspace.  Bound by HBM (6 D bytes per token and head).
#include "pkv_kernels.h"
#include "pkv_ptx.cuh"
#include "pkv_quant.cuh"
#include "pkv_scaled.h"

namespace pkv {

constexpr int kSsThreads = 256;
constexpr int kScaleLow = -40, kScaleHigh = 40;

// Bits of the largest finite magnitude of eight bf16 values (0 where there is none).
__device__ __forceinline__ uint32_t finite_max8(uint4 w)
{
    constexpr uint32_t ABS = 0x7fff7fffu;
    uint32_t m = bf16x2_max(bf16x2_max(w.x & ABS, w.y & ABS), bf16x2_max(w.z & ABS, w.w & ABS));
    m = max(m & 0xffffu, m >> 16);
    if (m >= 0x7f80u) {  // infinities, or nothing but NaN in a place of all four
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t lo = v[i] & 0x7fffu, hi = (v[i] >> 16) & 0x7fffu;
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

// T: tokens per window.  HOLD: row loads a thread keeps.
template <int D, int T, int HOLD>
__global__ void __launch_bounds__(kSsThreads) store_scaled_kernel(const StoreScaledParams p)
{
    constexpr int LPR = D / 8;              // lanes per row (16-byte loads)
    constexpr int RPP = kSsThreads / LPR;   // rows per pass
    static_assert(T <= kSsThreads - 1, "one thread per token of the window and one beyond");
    __shared__ int s_run[T];                // run of each token of the window, -1: none that starts here
    __shared__ int s_blk[T];
    __shared__ uint32_t s_max[T], s_begun[T];
    __shared__ float s_inv[T], s_ratio[T];
    __shared__ int s_grown[T];
    __shared__ uint32_t s_starts[kSsThreads / 32];
    __shared__ int s_more, s_n_grown;
    __shared__ long long s_end;

    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, z = blockIdx.z;
    const long long w0 = (long long)blockIdx.x * T;
    const uint32_t bs = (uint32_t)p.bs;

    // ---- the window's runs
    const auto slot_at = [&](long long i) -> long long { return i >= 0 && i < p.N ? __ldg(p.slots + i) : -1; };
    const auto block_of = [&](long long s) -> int {
        return s >= 0 && s < p.n_slots ? (int)((uint32_t)s / bs) : -1;
    };
    long long slot = -1;
    int blk = -1;
    bool start = false;
    if (tid <= T) {
        slot = slot_at(w0 + tid);
        blk = block_of(slot);
        const bool follows = blk >= 0 && block_of(slot_at(w0 + tid - 1)) == blk;
        start = tid < T && blk >= 0 && !follows;
        if (tid == T)
            s_more = follows;  // the last run goes on behind the window
        else if (slot != -1 && blk < 0 && h == 0 && z == 0)
            flag_error(p.err_flag, 0x1 /* PKV_FLAG_BAD_SLOT */);
    }
    if (tid < T)
        s_max[tid] = s_begun[tid] = 0;
    if (tid == 0)
        s_n_grown = 0;
    const uint32_t starts = __ballot_sync(0xffffffffu, start);
    if (lane == 0)
        s_starts[warp] = starts;
    __syncthreads();
    int before = 0, n_runs = 0, first = T;
#pragma unroll
    for (int i = 0; i < (T + 31) / 32; i++) {
        const uint32_t s = s_starts[i];
        before += i < warp ? __popc(s) : 0;
        n_runs += __popc(s);
        if (s && first == T)
            first = 32 * i + __ffs(s) - 1;
    }
    if (n_runs == 0) {
        // (a step of nothing but padding must not end before the kernel ahead of it)
        grid_dependency_wait();
        return;
    }
    if (tid < T) {
        const int run = blk >= 0 ? before + __popc(starts & (0xffffffffu >> (31 - lane))) - 1 : -1;
        s_run[tid] = run;
        if (start)
            s_blk[run] = blk;
        if (run >= 0 && (uint32_t)slot % bs == 0)
            s_begun[run] = 1;
    }
    if (tid == 0)
        s_end = w0 + T < p.N ? w0 + T : p.N;
    __syncthreads();
    if (s_more) {  // (the token behind the window lies in the last run's block)
        const int last = s_blk[n_runs - 1];
        for (long long i = w0 + T + tid;; i += kSsThreads) {
            const long long s = slot_at(i);
            const bool mine = block_of(s) == last;
            if (mine && (uint32_t)s % bs == 0)
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
        __syncthreads();
    }

    // ---- each run's largest magnitude; row i is token w0 + first + i
    const long long row0 = w0 + first;
    const long long rows = s_end - row0;
    const int sub = tid / LPR, part = tid % LPR;
    const auto run_of = [&](long long i) { return first + i < T ? s_run[first + i] : n_runs - 1; };
    const uint4 *src = (z ? p.x[1] : p.x[0]) + (row0 * p.Hkv + h) * LPR + part;
    const size_t stride = (size_t)p.Hkv * LPR;
    uint4 held[HOLD];
#pragma unroll
    for (int u = 0; u < HOLD; u++) {
        const long long i = u * RPP + sub;
        held[u] = make_uint4(0u, 0u, 0u, 0u);
        if (i < rows)
            held[u] = __ldg(src + i * stride);
    }
    const auto note = [&](uint4 w, long long i) {  // by all lanes of a warp
        uint32_t m = finite_max8(w);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (part == 0 && i < rows) {
            const int run = run_of(i);
            if (run >= 0)
                atomicMax(&s_max[run], m);
        }
    };
#pragma unroll
    for (int u = 0; u < HOLD; u++)
        if (u * RPP < rows)
            note(held[u], u * RPP + sub);
    for (long long i0 = HOLD * RPP; i0 < rows; i0 += RPP)
        note(i0 + sub < rows ? __ldg(src + (i0 + sub) * stride) : make_uint4(0u, 0u, 0u, 0u), i0 + sub);
    grid_dependency_wait();  // earlier kernels may still read the cache, or have written the scales
    __syncthreads();

    // ---- the scales
    if (tid < n_runs) {
        float *at = (z ? p.scales[1] : p.scales[0]) + (size_t)s_blk[tid] * p.Hkv + h;
        const float had = ld_gpu(at), want = scale_for(s_max[tid]);
        const bool keep = !s_begun[tid] && had > 0.f && had < INFINITY;
        const float now = keep ? fmaxf(had, want) : want;
        s_inv[tid] = __frcp_rn(now);
        if (!keep || now != had)
            *at = now;
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
            for (uint32_t c = tid; c < bs * CPR; c += kSsThreads) {
                uint4 *w = reinterpret_cast<uint4 *>(base + (size_t)(c / CPR) * p.Hkv * D + (c % CPR) * 16);
                const uint4 a = *w;
                *w = make_uint4(recode4(a.x, ratio), recode4(a.y, ratio), recode4(a.z, ratio),
                                recode4(a.w, ratio));
            }
        }
        __syncthreads();  // before rows of the same blocks are written over it
    }

    // ---- the rows
    const auto put = [&](uint4 w, long long i) {
        const int run = run_of(i);
        if (run < 0)
            return;
        const long long s = __ldg(p.slots + row0 + i);
        *reinterpret_cast<uint2 *>(cache + ((size_t)s * p.Hkv + h) * D + part * 8) = quantize8(w, s_inv[run]);
    };
#pragma unroll
    for (int u = 0; u < HOLD; u++)
        if (u * RPP + sub < rows)
            put(held[u], u * RPP + sub);
    for (long long i = HOLD * RPP + sub; i < rows; i += RPP)
        put(__ldg(src + i * stride), i);
}

template <int D> static cudaError_t launch(const StoreScaledParams &p, cudaStream_t stream)
{
    // Few tokens (decode steps: a run each): small windows, so that more CTAs share
    // them.  Many: windows of 128, of which a thread keeps 256 rows' loads in flight.
    const bool few = p.N < 2048;
    const int T = few ? 16 : 128;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((p.N + T - 1) / T), (unsigned)p.Hkv, 2);
    cfg.blockDim = dim3(kSsThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, store_scaled_kernel<D, 16, 2>, p)
               : cudaLaunchKernelEx(&cfg, store_scaled_kernel<D, 128, D / 8>, p);
}

cudaError_t launch_store_scaled(int D, const StoreScaledParams &p, cudaStream_t stream)
{
    return D == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

} // namespace pkv
