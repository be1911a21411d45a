// Decode attention that also says how much weight each cached token got.
//
//   out[b][h]      = softmax_p(scale * q[b][h] . K_b[p]) V_b[p]          (decode.cu)
//   scores[b][g][p] = (p < len - 1 ? scores_in : 0) + sum_{h in g} softmax weight of p
//
// The weights need the row's whole sum, which is known only when its last
// block has been read, and a second pass over K would cost half of the
// decode's traffic again.  So the decode unit leaves each token's score
// s = scale * log2(e) * q.k (fp32, 4 bytes a query head beside the 4 d bytes
// of a KV head's K and V) in a workspace and the row's log-sum-exp; the
// kernel below turns them into 2^(s - lse), sums over the KV head's query
// heads in a fixed order and adds.  The workspace is read back while most of
// it is in L2 (K and V are loaded evict-first).  (Adding inside the unit when
// it is done, to save the launch, took the single pass from 223 to 235 us at
// 256 sequences: 128 threads a CTA wait for L2 where they could stream K and V.)
// Measured: 256 sequences of 512 to 4096 tokens, 28/4 heads: the units 194 us (183
// without scores: the logits of 609 thousand tokens and 4 KV heads, 68 MB, 78 as
// stored with 7 heads padded to 8), this kernel 18; 8 x 32768, 32/8 heads: 162 + the
// merge's 7 + 10.  The workspace has a place for every token of every table, and the
// grid of this kernel a CTA for every 512 of them: both go by the tables' width.
#include "decode_unit.cuh"

namespace pkv {

namespace {

using namespace dev;

template <int D, bool MMA, int MODE>
__global__ void __launch_bounds__(128)
    paged_decode_scored_kernel(const __grid_constant__ CUtensorMap tmk,
                               const __grid_constant__ CUtensorMap tmv, const DecodeParams p) {
    if (p.order != nullptr) {
        pdl_wait_primary();
        decode_unit<D, 4, 2, MMA, MODE, true>(tmk, tmv, p, blockIdx.x, blockIdx.y, p.order[blockIdx.z]);
    } else {
        decode_unit<D, 4, 2, MMA, MODE, true>(tmk, tmv, p, blockIdx.x, blockIdx.y, static_cast<int>(blockIdx.z), true);
    }
}

// A thread's tokens of one (sequence, KV head): t0, t0 + kAddThreads, ...  Every
// load is issued before any is used; the logits of a block that was not read are
// loaded too (the workspace holds a place for every table entry) and left out.
constexpr int kAddThreads = 256;
constexpr int kAddTokens = 2;

template <int V>  // logits of a load: 4 where the width is a multiple of it, else 1
__global__ void __launch_bounds__(kAddThreads) score_add_kernel(const DecodeParams p, const ScoreParams sp) {
    pdl_launch_dependents();
    const int g = blockIdx.y, b = blockIdx.z;
    const int t0 = blockIdx.x * (kAddThreads * kAddTokens) + threadIdx.x;
    int len = __ldg(p.seq_lens + b);
    len = len < 0 ? 0 : min(len, p.W * kBlockTokens);
    bool live[kAddTokens];
    int32_t phys[kAddTokens];
#pragma unroll
    for (int i = 0; i < kAddTokens; ++i) {
        const int t = t0 + i * kAddThreads;
        live[i] = t < len;
        phys[i] = live[i] ? __ldg(p.block_tables + static_cast<size_t>(b) * p.W + t / kBlockTokens) : -1;
    }
    pdl_wait_primary();  // the lengths and tables are host-written; the rest is the grids' before
    if (blockIdx.x * (kAddThreads * kAddTokens) >= static_cast<unsigned>(len)) return;
    const size_t row = (static_cast<size_t>(b) * p.Hkv + g);
    const size_t at = row * sp.stride + t0;
    float before[kAddTokens], w[kAddTokens];
#pragma unroll
    for (int i = 0; i < kAddTokens; ++i) {
        before[i] = sp.scores_in != nullptr && t0 + i * kAddThreads < len - 1 ? sp.scores_in[at + i * kAddThreads] : 0.f;
        w[i] = 0.f;
    }
    const size_t tokens = static_cast<size_t>(p.W) * kBlockTokens;
    for (int c = 0; c < p.chunks; ++c) {
        const int heads = min(8, p.group - 8 * c);
        const float *lse = p.lse + static_cast<size_t>(b) * p.Hq + g * p.group + 8 * c;
        const float *s = p.logits + ((row * p.chunks + c) * tokens + t0) * p.logit_width;
#pragma unroll
        for (int h = 0; h < 8; h += V) {
            if (h >= heads) break;
            float x[kAddTokens][V];
#pragma unroll
            for (int i = 0; i < kAddTokens; ++i) {
                const float *src = s + static_cast<size_t>(i) * kAddThreads * p.logit_width + h;
                if constexpr (V == 4) {
                    const float4 v = live[i] ? __ldcg(reinterpret_cast<const float4 *>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[i][0] = v.x;
                    x[i][1] = v.y;
                    x[i][2] = v.z;
                    x[i][3] = v.w;
                } else {
                    x[i][0] = live[i] ? __ldcg(src) : 0.f;
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (h + e >= heads) break;
                const float l = lse[h + e];
#pragma unroll
                for (int i = 0; i < kAddTokens; ++i) w[i] += ex2_approx(x[i][e] - l);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kAddTokens; ++i)
        if (live[i])
            sp.scores_out[at + i * kAddThreads] = before[i] + (phys[i] >= 0 && phys[i] < p.num_blocks ? w[i] : 0.f);
}

template <int D, bool MMA, int MODE>
cudaError_t launch_one(const CUtensorMap &tmk, const CUtensorMap &tmv, const DecodeParams &p, cudaStream_t stream) {
    using G = Geometry<D, 4, 2>;
    constexpr int kSmem = G::kSmemBytes + (MODE == kModeCluster ? cluster_land_bytes<D, MMA>() : 0);
    auto kern = paged_decode_scored_kernel<D, MMA, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_parts), static_cast<unsigned>(MMA ? p.Hkv * p.chunks : p.Hq),
                       static_cast<unsigned>(p.B));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
    if (MODE == kModeCluster) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(p.num_parts);
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    e = cudaLaunchKernelEx(&cfg, kern, tmk, tmv, p);
    if (e != cudaSuccess || MODE != kModeSplit) return e;
    return launch_splitk_merge(p, D, stream);
}

template <int D, bool MMA>
cudaError_t launch_m(const CUtensorMap &tmk, const CUtensorMap &tmv, const DecodeParams &p, int mode,
                     cudaStream_t stream) {
    if (mode == kModeSplit) return launch_one<D, MMA, kModeSplit>(tmk, tmv, p, stream);
    if (mode == kModeCluster) return launch_one<D, MMA, kModeCluster>(tmk, tmv, p, stream);
    return launch_one<D, MMA, kModeSingle>(tmk, tmv, p, stream);
}

}  // namespace

cudaError_t launch_decode_scored(const CUtensorMap &tmk, const CUtensorMap &tmv, const DecodeParams &p,
                                 const ScoreParams &sp, int head_dim, int mode, cudaStream_t stream) {
    cudaError_t e = cudaErrorInvalidValue;
    if (mode == kModeCluster && (p.num_parts < 1 || p.num_parts > kMaxClusterParts)) return e;
    if (head_dim == 128)
        e = p.group > 1 ? launch_m<128, true>(tmk, tmv, p, mode, stream)
                        : launch_m<128, false>(tmk, tmv, p, mode, stream);
    else if (head_dim == 64)
        e = p.group > 1 ? launch_m<64, true>(tmk, tmv, p, mode, stream)
                        : launch_m<64, false>(tmk, tmv, p, mode, stream);
    if (e != cudaSuccess) return e;
    constexpr int kTokens = kAddThreads * kAddTokens;
    const unsigned gx = static_cast<unsigned>((static_cast<long long>(p.W) * kBlockTokens + kTokens - 1) / kTokens);
    return launch_dependent(p.logit_width % 4 == 0 ? score_add_kernel<4> : score_add_kernel<1>,
                            dim3(gx, static_cast<unsigned>(p.Hkv), static_cast<unsigned>(p.B)), dim3(kAddThreads),
                            stream, p, sp);
}

}  // namespace pkv
