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
// evict_select_kernel: a cluster of 1 to 4 CTAs per (sequence, KV head), each
// CTA a slice of its tokens, finds the m-th largest of order-preserving integer
// keys (the tokens that stay anyway hold the largest key) by a radix select:
// 8 bits a pass, a histogram in each CTA's shared memory, the cluster's sum
// read through distributed shared memory.  One ordered pass then writes the
// kept positions: every key above the threshold and the first of those equal
// to it.  No sort, and the result does not depend on the order of any atomic.
// evict_copy_kernel: the rows and their scores; bound by HBM (each kept row
// read and written once): 302 MB in 51 us, 268 MB in 42 us (5.9 and 6.3 TB/s).
#include <algorithm>

#include "decode_common.cuh"

namespace pkv {

namespace {

using namespace dev;

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
    e.len = p.seq_lens[b];
    int keep = p.keep_lens[b];
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

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kPer = 8;                     // consecutive tokens of a thread
constexpr int kRound = kSelThreads * kPer;  // tokens a CTA holds in registers: 4096
constexpr int kMaxSlices = 4;               // CTAs of a cluster
constexpr int kCopies = 4;

// Block-wide exclusive scan of x; *total gets the sum.
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
    for (int w = 0; w < kSelWarps; ++w) {
        const int v = warp_sums[w];
        before += w < warp ? v : 0;
        sum += v;
    }
    *total = sum;
    return before + incl - x;
}

// The keys of tokens [t0, t0 + kPer) of one row; the tokens that stay anyway
// hold the largest key, which no score has.
__device__ __forceinline__ void load_keys(const float *in, bool vec, int t0, const EvictRow &e, uint32_t (&k)[kPer]) {
    float x[kPer];
    if (vec && t0 + kPer <= e.len) {
        *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(in + t0);
        *reinterpret_cast<float4 *>(x + 4) = *reinterpret_cast<const float4 *>(in + t0 + 4);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = t0 + i < e.len ? in[t0 + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        k[i] = t0 + i < e.s || t0 + i >= e.len - e.r ? 0xFFFFFFFFu : score_key(x[i]);
}

// A few microseconds of barriers and first executions: 8 keys a thread stay in
// registers (a round; longer slices read theirs again each pass).  For 256 rows
// of about 2300 scores it takes 10 us, with 16 keys unrolled 17, with the keys
// in shared memory 14; for 64 rows of 32768, four CTAs a row take 23 us (22 when
// the other figures here were taken: with 16 keys 23.5, though none is read twice,
// two CTAs 32 and eight 27 -- their five cluster barriers --, one with all keys in
// shared memory 38).
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p, int slices) {
    pdl_launch_dependents();
    // A pass counts into kCopies histograms, a lane into its own (scores share few
    // leading bytes, and a warp's updates of one word go one after another), ...
    __shared__ __align__(16) int spread[256 * kCopies];
    __shared__ int hist[4][256];  // ... summed here; one per pass: another CTA may still read the last pass's
    __shared__ int warp_sums[kSelWarps];
    __shared__ int found[2];      // the pass's bin, the keys above it
    __shared__ int counts[2];     // this slice's keys above and at the threshold
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int h = blockIdx.y, b = blockIdx.z;
    const auto clear = [&] {
        for (int i = tid; i < 256 * kCopies / 4; i += kSelThreads) reinterpret_cast<int4 *>(spread)[i] = make_int4(0, 0, 0, 0);
    };
    clear();
    pdl_wait_primary();
    bool bad;
    const EvictRow e = evict_row(p, b, &bad);
    if (bad && h == 0 && rank == 0 && tid == 0) flag(p.err, PKV_DEV_ERR_BAD_LEN);
    const size_t row = static_cast<size_t>(b) * p.Hkv + h;
    const float *in = p.scores_in + row * p.in_stride;
    int32_t *kept = p.kept + row * (static_cast<size_t>(p.NW) * kBlockTokens);
    // this CTA's tokens [lo, hi), lo a multiple of kPer (whole cluster: the same e)
    const int per = ((e.len + slices - 1) / slices + kPer - 1) / kPer * kPer;
    const int lo = min(rank * per, e.len), hi = min(lo + per, e.len);
    if (e.m == e.len || e.m == 0) {  // nothing goes, or everything
        if (e.m > 0)
            for (int t = lo + tid; t < hi; t += kSelThreads) kept[t] = t;
        return;
    }
    const bool vec = (reinterpret_cast<uintptr_t>(in) & 15u) == 0;
    const int rounds = (per + kRound - 1) / kRound;
    uint32_t k0[kPer];
    load_keys(in, vec, lo + tid * kPer, e, k0);
    __syncthreads();  // cleared
    uint32_t prefix = 0;  // the m-th largest key's bits so far
    int need = e.m;       // its rank among the keys that share them
    bool all = false;     // every key that shares them is kept
#pragma unroll 1
    for (int pass = 0; pass < 4 && !all; ++pass) {
        const int shift = 24 - 8 * pass;
        const uint32_t mask = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
#pragma unroll 1
        for (int r = 0; r < rounds; ++r) {
            const int t0 = lo + r * kRound + tid * kPer;
            uint32_t k[kPer];
            if (r == 0) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) k[i] = k0[i];
            } else {
                load_keys(in, vec, t0, e, k);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (t0 + i < hi && (k[i] & mask) == prefix)
                    atomicAdd(&spread[((k[i] >> shift) & 255) * kCopies + lane % kCopies], 1);
        }
        __syncthreads();
        int mine = 0;  // thread i < 256: this slice's, then the cluster's count of bin 255 - i
        if (tid < 256) {
#pragma unroll
            for (int i = 0; i < kCopies; i += 4) {
                const int4 v = *reinterpret_cast<const int4 *>(spread + (255 - tid) * kCopies + i);
                mine += (v.x + v.y) + (v.z + v.w);
            }
            hist[pass][255 - tid] = mine;
        }
        if (slices > 1) {
            cluster_arrive_release();
            cluster_wait_acquire();
            if (tid < 256) {
                const uint32_t at = smem_u32(&hist[pass][255 - tid]);
                mine = 0;
#pragma unroll
                for (int c = 0; c < kMaxSlices; ++c)
                    if (c < slices) mine += static_cast<int>(ld_dsmem_u32(dsmem_addr(at, c)));
            }
        }
        // the keys in the bins above
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();  // and: this pass's copies are read
        clear();
        if (tid < 256) {
            int above = incl - mine;
#pragma unroll
            for (int w = 0; w < 8; ++w) above += w < warp ? warp_sums[w] : 0;
            if (above < need && need <= above + mine) {  // exactly one thread
                found[0] = (255 - tid) | (need == above + mine ? 256 : 0);
                found[1] = above;
            }
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(found[0] & 255) << shift;
        need -= found[1];
        // every key of the bin is kept: the remaining bits need no telling apart
        all = (found[0] & 256) && prefix != 0;
    }
    // kept: keys above the threshold, and the first `need` equal to it
    const uint32_t threshold = all ? prefix - 1 : prefix;
    if (all) need = 0;
    // this slice's first place: the keys above and at the threshold in the slices before it
    int above0 = 0, equal0 = 0;
    const auto count = [&](const uint32_t (&k)[kPer], int t0) {
        int n = 0;  // keys above the threshold, and (from bit 16) equal to it: at most kRound of each
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (t0 + i < hi) n += k[i] > threshold ? 1 : k[i] == threshold ? 1 << 16 : 0;
        return n;
    };
    int total0, packed0 = block_scan(count(k0, lo + tid * kPer), warp_sums, &total0);
    if (slices > 1) {
        int above = total0 & 0xFFFF, equal = total0 >> 16;
#pragma unroll 1
        for (int r = 1; r < rounds; ++r) {
            const int t0 = lo + r * kRound + tid * kPer;
            uint32_t k[kPer];
            load_keys(in, vec, t0, e, k);
            int total;
            block_scan(count(k, t0), warp_sums, &total);
            above += total & 0xFFFF;
            equal += total >> 16;
        }
        if (tid == 0) {
            counts[0] = above;
            counts[1] = equal;
        }
        cluster_arrive_release();
        cluster_wait_acquire();
#pragma unroll
        for (int c = 0; c < kMaxSlices - 1; ++c)
            if (c < rank) {
                above0 += static_cast<int>(ld_dsmem_u32(dsmem_addr(smem_u32(&counts[0]), c)));
                equal0 += static_cast<int>(ld_dsmem_u32(dsmem_addr(smem_u32(&counts[1]), c)));
            }
        cluster_arrive_release();  // this CTA reads no other's memory from here on
    }
    // a kept token's place: those kept before it
#pragma unroll 1
    for (int r = 0; r < rounds; ++r) {
        const int t0 = lo + r * kRound + tid * kPer;
        uint32_t k[kPer];
        int total = total0, packed = packed0;
        if (r == 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) k[i] = k0[i];
        } else {
            load_keys(in, vec, t0, e, k);
            packed = block_scan(count(k, t0), warp_sums, &total);
        }
        int a = above0 + (packed & 0xFFFF), q = equal0 + (packed >> 16);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (t0 + i < hi) {
                const bool gt = k[i] > threshold, eq = k[i] == threshold;
                if (gt || (eq && q < need)) kept[a + min(q, need)] = t0 + i;
                a += gt;
                q += eq;
            }
        }
        above0 += total & 0xFFFF;
        equal0 += total >> 16;
    }
    if (slices > 1) cluster_wait_acquire();  // the others have read this CTA's counts
}

constexpr int kCopyThreads = 256;
constexpr int kGroup = 32;  // kept tokens of a warp, one lane each for their addresses

// A warp moves 32 kept tokens; a pass of it one row of K and one of V (D = 128:
// half a warp each) or two of both, kBatch passes' loads in flight.  Many warps
// with few rows each, not few with many: the addresses are three loads that
// wait for one another (length, kept position, table entry), and warps in
// their copy hide those of the next.
template <int D>
__global__ void __launch_bounds__(kCopyThreads, 4) evict_copy_kernel(const EvictParams p) {
    pdl_launch_dependents();
    constexpr int kVec = D / 8;             // 16-byte vectors of a row
    constexpr int kRows = 32 / (2 * kVec);  // tokens of one pass
    constexpr int kBatch = 8;
    static_assert(kGroup == 32 && kGroup % (kBatch * kRows) == 0, "one lane per token");
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y, b = blockIdx.z;
    const int first = (blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5)) * kGroup;
    pdl_wait_primary();
    bool bad;
    const EvictRow e = evict_row(p, b, &bad);
    if (first >= e.m) return;
    const int i = first + lane;
    int src = -1, dst = -1;  // rows of the caches (num_blocks * Hkv * 16 < 2^31), -1: none
    if (i < e.m) {
        const size_t row = static_cast<size_t>(b) * p.Hkv + h;
        const int t = __ldcg(p.kept + row * (static_cast<size_t>(p.NW) * kBlockTokens) + i);
        const int32_t to = p.new_tables[static_cast<size_t>(b) * p.NW + i / kBlockTokens];
        const int32_t from = p.block_tables[static_cast<size_t>(b) * p.W + t / kBlockTokens];
        p.scores_out[row * p.out_stride + i] = p.scores_in[row * p.in_stride + t];
        if (from >= 0 && from < p.num_blocks && to >= 0 && to < p.num_blocks) {
            src = (from * p.Hkv + h) * kBlockTokens + t % kBlockTokens;
            dst = (to * p.Hkv + h) * kBlockTokens + i % kBlockTokens;
        } else {
            flag(p.err, PKV_DEV_ERR_BAD_BLOCK);
        }
    }
    const int sub = lane / (2 * kVec);  // which token of a pass
    const bool is_v = (lane / kVec) & 1;
    uint4 *cache = reinterpret_cast<uint4 *>(is_v ? p.v_cache : p.k_cache) + lane % kVec;
#pragma unroll
    for (int i0 = 0; i0 < kGroup; i0 += kBatch * kRows) {
        uint4 x[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int from = __shfl_sync(0xffffffffu, src, i0 + j * kRows + sub);
            if (from >= 0) x[j] = __ldcs(cache + static_cast<long long>(from) * kVec);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int to = __shfl_sync(0xffffffffu, dst, i0 + j * kRows + sub);
            if (to >= 0) cache[static_cast<long long>(to) * kVec] = x[j];
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int head_dim, cudaStream_t stream) {
    // a CTA for each kRound tokens of the longest row, at most kMaxSlices
    const long long tokens = static_cast<long long>(p.W) * kBlockTokens;
    int slices = 1;
    while (slices < kMaxSlices && static_cast<long long>(slices) * kRound < tokens) slices *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(slices), static_cast<unsigned>(p.Hkv), static_cast<unsigned>(p.B));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(slices);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = slices > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, slices);
    if (e != cudaSuccess) return e;
    const long long most = static_cast<long long>(p.NW) * kBlockTokens;
    constexpr int kTokens = kCopyThreads / 32 * kGroup;  // of a CTA
    const dim3 grid(static_cast<unsigned>((most + kTokens - 1) / kTokens), static_cast<unsigned>(p.Hkv),
                    static_cast<unsigned>(p.B));
    return launch_dependent(head_dim == 128 ? evict_copy_kernel<128> : evict_copy_kernel<64>, grid, dim3(kCopyThreads),
                            stream, p);
}

}  // namespace pkv
