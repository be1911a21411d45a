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
// heads in a fixed order and adds.
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
        decode_unit<D, 4, 2, MMA, MODE, true>(tmk, tmv, p, blockIdx.x, blockIdx.y,
                                              __ldg(p.order + blockIdx.z));
    } else {
        decode_unit<D, 4, 2, MMA, MODE, true>(tmk, tmv, p, blockIdx.x, blockIdx.y,
                                              static_cast<int>(blockIdx.z), true);
    }
}

// One thread per (sequence, KV head, token).
constexpr int kAddThreads = 256;

__global__ void __launch_bounds__(kAddThreads)
    score_add_kernel(const DecodeParams p, const ScoreParams sp) {
    pdl_launch_dependents();
    const int g = blockIdx.y, b = blockIdx.z;
    const int t = blockIdx.x * kAddThreads + threadIdx.x;
    pdl_wait_primary();
    int len = __ldg(p.seq_lens + b);
    len = len < 0 ? 0 : min(len, p.W * kBlockTokens);
    if (t >= len) return;
    const size_t tokens = static_cast<size_t>(p.W) * kBlockTokens;
    const int32_t phys = __ldg(p.block_tables + static_cast<size_t>(b) * p.W + t / kBlockTokens);
    float w = 0.f;
    if (phys >= 0 && phys < p.num_blocks) {  // a block that was not read has no weight
        for (int c = 0; c < p.chunks; ++c) {
            const float *s = p.logits +
                             (((static_cast<size_t>(b) * p.Hkv + g) * p.chunks + c) * tokens + t) * p.logit_width;
            const float *lse = p.lse + static_cast<size_t>(b) * p.Hq + g * p.group + 8 * c;
            const int heads = min(8, p.group - 8 * c);
#pragma unroll
            for (int h = 0; h < 8; ++h)
                if (h < heads) w += ex2_approx(s[h] - lse[h]);
        }
    }
    const size_t at = (static_cast<size_t>(b) * p.Hkv + g) * sp.stride + t;
    const float before = sp.scores_in != nullptr && t < len - 1 ? sp.scores_in[at] : 0.f;
    sp.scores_out[at] = before + w;
}

template <int D, bool MMA, int MODE>
cudaError_t launch_one(const CUtensorMap &tmk, const CUtensorMap &tmv, const DecodeParams &p,
                       cudaStream_t stream) {
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
    const unsigned gx = static_cast<unsigned>((static_cast<long long>(p.W) * kBlockTokens + kAddThreads - 1) / kAddThreads);
    return launch_dependent(score_add_kernel, dim3(gx, static_cast<unsigned>(p.Hkv), static_cast<unsigned>(p.B)),
                            dim3(kAddThreads), stream, p, sp);
}

}  // namespace pkv
