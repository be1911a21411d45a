// Eviction by accumulated attention weight.
//
// For each (sequence, KV head): of the cached tokens [0, len) keep m =
// min(keep_lens[b], len) -- the last r = min(recent, m), the first
// s = min(sink, m - r), and of the others the m - r - s with the highest
// scores (equal scores: the lower position; NaN counts as lowest) -- and copy
// their K, V and scores, in position order, to positions [0, m) of the
// sequence's new table.  Keys carry their rotation already, so a token may
// sit anywhere.  The old blocks are only read: they may be shared.
//
// evict_select_kernel: one CTA per (sequence, KV head) finds the
// (m - r - s)-th largest score by a radix select over order-preserving
// integer keys (11 + 11 + 10 bits, a histogram in shared memory each), then
// one ordered pass writes the kept positions: every key above the threshold
// and the first of those equal to it.  No sort, and the result does not depend
// on the order of any atomic.
// evict_copy_kernel: the rows; bound by HBM (each kept row read and written
// once).
#include <algorithm>

#include "decode_common.cuh"

namespace pkv {

namespace {

using namespace dev;

constexpr int kStagedTokens = 48 * 1024;  // keys kept in shared memory up to here (192 KB)

// Larger key = higher score.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0u;  // NaN: below -inf (0x007FFFFF)
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Lengths of one sequence: tokens, kept, of them recent and sink.
struct EvictRow {
    int len, m, r, s;
};
__device__ __forceinline__ EvictRow evict_row(const EvictParams &p, int b, bool *bad) {
    EvictRow e;
    e.len = __ldg(p.seq_lens + b);
    int keep = __ldg(p.keep_lens + b);
    const long long cap = static_cast<long long>(p.W) * kBlockTokens;
    const long long new_cap = static_cast<long long>(p.NW) * kBlockTokens;
    *bad = e.len < 0 || e.len > cap || keep < 0;
    e.len = static_cast<int>(min(static_cast<long long>(max(e.len, 0)), cap));
    keep = min(max(keep, 0), e.len);
    if (keep > new_cap) {
        *bad = true;
        keep = static_cast<int>(new_cap);
    }
    e.m = keep;
    e.r = min(p.recent, e.m);
    e.s = min(p.sink, e.m - e.r);
    return e;
}

// Block-wide exclusive scan of x over THREADS threads; *total gets the sum.
template <int THREADS>
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    __syncthreads();  // warp_sums of the previous scan are read
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const int v = warp_sums[w];
        before += w < warp ? v : 0;
        sum += v;
    }
    *total = sum;
    return before + incl - x;
}

constexpr int kBins = 2048;
constexpr int kPerThread = 4;  // consecutive tokens a thread takes in the ordered pass

template <int THREADS, bool STAGED>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const EvictParams p) {
    pdl_launch_dependents();
    extern __shared__ uint32_t keys[];  // [len] when STAGED
    __shared__ int hist[kBins];
    __shared__ int warp_sums[THREADS / 32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    pdl_wait_primary();
    bool bad;
    const EvictRow e = evict_row(p, b, &bad);
    if (bad && h == 0 && tid == 0) flag(p.err, PKV_DEV_ERR_BAD_LEN);
    const size_t row = static_cast<size_t>(b) * p.Hkv + h;
    const float *in = p.scores_in + row * p.in_stride;
    float *out = p.scores_out + row * p.out_stride;
    int32_t *kept = p.kept + row * (static_cast<size_t>(p.NW) * kBlockTokens);
    if (e.m == e.len) {  // nothing goes
        for (int t = tid; t < e.len; t += THREADS) {
            kept[t] = t;
            out[t] = in[t];
        }
        return;
    }
    const int lo = e.s, hi = e.len - e.r;  // the tokens that compete
    const int want = e.m - e.r - e.s;      // 0 <= want < hi - lo
    if (STAGED) {
        for (int t = lo + tid; t < hi; t += THREADS) keys[t] = score_key(__ldg(in + t));
    }
    const auto key_at = [&](int t) { return STAGED ? keys[t] : score_key(__ldg(in + t)); };
    // the want-th largest key: `prefix` its bits so far, `need` its rank among
    // the keys that share them
    uint32_t prefix = 0;
    int need = want;
    if (want > 0) {
        if (tid == 0) {
            s_prefix = 0;
            s_need = want;
        }
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bits = pass == 2 ? 10 : 11;
            const uint32_t mask = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + bits);
            for (int i = tid; i < kBins; i += THREADS) hist[i] = 0;
            __syncthreads();  // also: keys staged, s_prefix and s_need written
            prefix = s_prefix;
            need = s_need;
            for (int t = lo + tid; t < hi; t += THREADS) {
                const uint32_t k = key_at(t);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
            }
            __syncthreads();
            // bins from the top: thread i owns the kBins / THREADS bins below those of thread i - 1
            constexpr int kOwn = kBins / THREADS;
            int own[kOwn], sum = 0;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                own[i] = hist[kBins - 1 - (tid * kOwn + i)];
                sum += own[i];
            }
            int total;
            int above = block_scan<THREADS>(sum, warp_sums, &total);
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                if (above < need && need <= above + own[i]) {  // exactly one bin of one thread
                    s_prefix = prefix | (static_cast<uint32_t>(kBins - 1 - (tid * kOwn + i)) << shift);
                    s_need = need - above;
                }
                above += own[i];
            }
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
    } else {
        __syncthreads();
    }
    // In position order: sinks, keys above the threshold and the first `need`
    // equal to it, recent tokens.  A token's place = the kept ones before it.
    for (int t = tid; t < e.s; t += THREADS) {
        kept[t] = t;
        out[t] = in[t];
    }
    for (int t = hi + tid; t < e.len; t += THREADS) {
        const int i = e.m - (e.len - t);
        kept[i] = t;
        out[i] = in[t];
    }
    if (want == 0) return;
    int above_before = 0, equal_before = 0;
    for (int base = lo; base < hi; base += THREADS * kPerThread) {
        const int t0 = base + tid * kPerThread;
        uint32_t k[kPerThread];
        int n_above = 0, n_equal = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            k[i] = t0 + i < hi ? key_at(t0 + i) : 0u;
            if (t0 + i < hi) {
                n_above += k[i] > prefix;
                n_equal += k[i] == prefix;
            }
        }
        // both counts in one scan: at most THREADS * kPerThread <= 4096 of each
        int total;
        const int packed = block_scan<THREADS>(n_above | (n_equal << 16), warp_sums, &total);
        int a = above_before + (packed & 0xFFFF), q = equal_before + (packed >> 16);
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int t = t0 + i;
            if (t < hi) {
                const bool gt = k[i] > prefix, eq = k[i] == prefix;
                if (gt || (eq && q < need)) {
                    const int at = e.s + a + min(q, need);
                    kept[at] = t;
                    out[at] = in[t];
                }
                a += gt;
                q += eq;
            }
        }
        above_before += total & 0xFFFF;
        equal_before += total >> 16;
    }
}

constexpr int kCopyThreads = 256;
constexpr int kWarpTokens = 32;  // kept tokens of one warp
constexpr int kCopyTokens = kCopyThreads / 32 * kWarpTokens;

// A warp moves one row of K (its first D / 8 lanes) and V (the next) at a
// time per 32 / (D / 4) tokens, 8 rows' loads in flight.
template <int D>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p) {
    pdl_launch_dependents();
    constexpr int kVec = D / 8;             // 16-byte vectors of a row
    constexpr int kRows = 32 / (2 * kVec);  // tokens of one pass (K and V)
    constexpr int kBatch = 8;
    static_assert(kWarpTokens == 32 && 32 % (kBatch * kRows) == 0, "one lane per token of the warp");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.y, b = blockIdx.z;
    pdl_wait_primary();
    bool bad;
    const EvictRow e = evict_row(p, b, &bad);
    const int first = blockIdx.x * kCopyTokens + warp * kWarpTokens;
    if (first >= e.m) return;
    const int n = min(kWarpTokens, e.m - first);
    // lane i: source and destination row of token first + i (-1: left out)
    long long src = -1, dst = -1;
    if (lane < n) {
        const int i = first + lane;
        const int t = __ldcg(p.kept + (static_cast<size_t>(b) * p.Hkv + h) * (static_cast<size_t>(p.NW) * kBlockTokens) + i);
        const int32_t from = __ldg(p.block_tables + static_cast<size_t>(b) * p.W + t / kBlockTokens);
        const int32_t to = __ldg(p.new_tables + static_cast<size_t>(b) * p.NW + i / kBlockTokens);
        if (from >= 0 && from < p.num_blocks && to >= 0 && to < p.num_blocks) {
            src = (static_cast<long long>(from) * p.Hkv + h) * kBlockTokens + t % kBlockTokens;
            dst = (static_cast<long long>(to) * p.Hkv + h) * kBlockTokens + i % kBlockTokens;
        } else {
            flag(p.err, PKV_DEV_ERR_BAD_BLOCK);
        }
    }
    const int sub = lane / (2 * kVec);  // which token of a pass
    const int vec = lane % kVec;
    const bool is_v = (lane / kVec) & 1;
    uint4 *cache = reinterpret_cast<uint4 *>(is_v ? p.v_cache : p.k_cache);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kBatch * kRows) {
        uint4 x[kBatch];
        long long to[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * kRows + sub;
            // (lanes at or past n hold -1)
            const long long from = __shfl_sync(0xffffffffu, src, i);
            to[j] = __shfl_sync(0xffffffffu, dst, i);
            if (from >= 0) x[j] = __ldcs(cache + from * kVec + vec);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (to[j] >= 0) cache[to[j] * kVec + vec] = x[j];
    }
}

template <int THREADS, bool STAGED>
cudaError_t launch_select(const EvictParams &p, size_t smem, cudaStream_t stream) {
    auto kern = evict_select_kernel<THREADS, STAGED>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_dependent_smem(kern, dim3(static_cast<unsigned>(p.Hkv), static_cast<unsigned>(p.B)), dim3(THREADS),
                                 smem, stream, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int head_dim, cudaStream_t stream) {
    const long long tokens = static_cast<long long>(p.W) * kBlockTokens;
    cudaError_t e;
    if (tokens <= 8192)
        e = launch_select<256, true>(p, static_cast<size_t>(tokens) * 4, stream);
    else if (tokens <= kStagedTokens)
        e = launch_select<1024, true>(p, static_cast<size_t>(tokens) * 4, stream);
    else
        e = launch_select<1024, false>(p, 0, stream);
    if (e != cudaSuccess) return e;
    const long long most = static_cast<long long>(p.NW) * kBlockTokens;
    const dim3 grid(static_cast<unsigned>((most + kCopyTokens - 1) / kCopyTokens), static_cast<unsigned>(p.Hkv),
                    static_cast<unsigned>(p.B));
    if (head_dim == 128) return launch_dependent(evict_copy_kernel<128>, grid, dim3(kCopyThreads), stream, p);
    if (head_dim == 64) return launch_dependent(evict_copy_kernel<64>, grid, dim3(kCopyThreads), stream, p);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
