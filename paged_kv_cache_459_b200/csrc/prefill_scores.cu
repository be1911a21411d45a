// The weight a chunk's queries put on each cached token, on tcgen05.
//
//   scores[b][g][p] = (p < first new position ? scores_in : 0)
//                     + sum over the counted new tokens t at positions >= p and the heads h of group g
//                       of 2^(scale log2(e) q[t][h].k[p] - lse[t][h])
// with lse the row's log-sum-exp that the prefill kernel left behind (log2
// domain), so one product Q K^T and no running maximum.
//
// The product is taken transposed: a work unit owns 128 keys (MMA rows, TMEM
// lanes) of one (sequence, KV head) and walks the counted queries that see
// them in tiles of 128 rows (columns), so a thread's sum over its lane's
// columns is the key's sum and nothing crosses threads.  The K tile stays in
// shared memory for the whole unit; Q tiles come by TMA as boxes of [tokens]
// [heads of the group][64] (128 / group tokens each; a group that does not
// divide 128 leaves zeroed rows).  S is double-buffered in TMEM and two CTAs
// share an SM, so that the products of one tile run behind the exponentials
// of another.  Bound by the exponentials: 128 x 128 of them take the
// special-function unit 1024 cycles, the tile's products 512.
// Few units (few sequences, short contexts): each unit's queries are cut into
// `splits` ranges whose sums a second kernel adds in order.
#include <algorithm>

#include "decode_common.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

using namespace dev;

constexpr int kKeys = 128;      // keys of a unit (MMA M)
constexpr int kCols = 128;      // query rows of a tile (MMA N)
constexpr int kExpWarps = 4;    // TMEM lanes 32 w .. 32 w + 31 belong to warp w
constexpr int kProducerWarp = 4, kMmaWarp = 5;
constexpr int kThreads = 192;
constexpr int kQStages = 2;
constexpr int kSBuffers = 2;

template <int D>
struct ScoreGeometry {
    static constexpr int kHalves = D / 64;
    static constexpr int kTileBytes = kHalves * 128 * 128;  // K tile or Q tile: [half][row][128 B]
    static constexpr int kQ = kTileBytes;                   // + stage * kTileBytes
    static constexpr int kNeg = kQ + kQStages * kTileBytes;  // -lse of the tile's rows, two buffers
    static constexpr int kBars = kNeg + 2 * kCols * 4;
    static constexpr int kNumBars = 1 + 2 * kQStages + 2 * kSBuffers;
    static constexpr int kTmemSlot = kBars + kNumBars * 8;
    static constexpr int kSmemBytes = kTmemSlot + 16 + 1024;
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

// One sequence's part in the scores.
struct ScoreSeq {
    int q0, nq, ctx, first_pos, first_tok;  // first_tok: first counted new token
};
// False for a sequence whose lengths do not fit (flagged by its first unit).
__device__ __forceinline__ bool score_seq(const PrefillScoreParams &p, int b, ScoreSeq &s) {
    s.q0 = __ldg(p.pp.query_start + b);
    s.nq = max(__ldg(p.pp.query_start + b + 1) - s.q0, 0);
    s.ctx = __ldg(p.pp.seq_lens + b);
    s.first_pos = s.ctx - s.nq;
    s.first_tok = max(0, s.nq - p.window);
    return s.first_pos >= 0 && s.ctx <= p.pp.W * kBlockTokens && s.nq <= p.max_query_len &&
           (s.nq == 0 || (s.q0 >= 0 && s.q0 <= p.pp.num_tokens - s.nq));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    prefill_scores_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmq,
                          const PrefillScoreParams p) {
    using Geo = ScoreGeometry<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / p.pp.Hkv, kvh = blockIdx.x % p.pp.Hkv;
    const int key_lo = blockIdx.y * kKeys, split = blockIdx.z;
    const int G = p.pp.group;

    ScoreSeq sq;
    if (!score_seq(p, b, sq)) {
        if (threadIdx.x == 0 && kvh == 0 && blockIdx.y == 0 && split == 0) flag(p.pp.err, PKV_DEV_ERR_BAD_LEN);
        return;
    }
    if (key_lo >= sq.ctx) return;
    // counted tokens that see some key of the unit, in tiles of tile_tokens; this CTA's range of tiles
    const int tok_lo = max(sq.first_tok, key_lo - sq.first_pos);
    const int all = sq.nq > tok_lo ? (sq.nq - tok_lo + p.tile_tokens - 1) / p.tile_tokens : 0;
    const int i0 = static_cast<int>(static_cast<long long>(all) * split / p.splits);
    const int i1 = static_cast<int>(static_cast<long long>(all) * (split + 1) / p.splits);
    const int n = i1 - i0;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float total = 0.f;
    if (n > 0) {
        const uint32_t bar0 = smem_u32(smem + Geo::kBars);
        const uint32_t k_full = bar0;
        const auto q_full = [&](int s) { return bar0 + 8 * (1 + s); };
        const auto q_empty = [&](int s) { return bar0 + 8 * (1 + kQStages + s); };
        const auto s_full = [&](int x) { return bar0 + 8 * (1 + 2 * kQStages + x); };
        const auto s_empty = [&](int x) { return bar0 + 8 * (1 + 2 * kQStages + kSBuffers + x); };
        uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Geo::kTmemSlot);
        volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Geo::kTmemSlot + 4);
        const int rows = p.tile_tokens * G;  // rows a Q box fills

        if (threadIdx.x == 0) {
            mbar_init(k_full, 1);
            for (int s = 0; s < kQStages; ++s) {
                mbar_init(q_full(s), 1);
                mbar_init(q_empty(s), 1);
            }
            for (int x = 0; x < kSBuffers; ++x) {
                mbar_init(s_full(x), 1);
                mbar_init(s_empty(x), kExpWarps);
            }
            *abort_flag = 0;
            fence_mbar_init();
            prefetch_tmap(&tmk);
            prefetch_tmap(&tmq);
        }
        // rows no box fills hold zeros: their scores are 0, their -lse is -inf
        for (int idx = threadIdx.x; idx < (kCols - rows) * Geo::kHalves * 8 * kQStages; idx += kThreads) {
            const int c = idx % 8, r = rows + idx / 8 % (kCols - rows), rest = idx / 8 / (kCols - rows);
            *reinterpret_cast<uint4 *>(smem + Geo::kQ + rest * (128 * 128) + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        if (warp == kMmaWarp) tc::alloc<kSBuffers * kCols>(smem_u32(tmem_slot));
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
        const uint32_t tmem = *tmem_slot;

        if (warp == kProducerWarp) {
            if (lane == 0) {
                const uint64_t policy = l2_policy_evict_normal();
                const int nblk = (sq.ctx + kBlockTokens - 1) / kBlockTokens;
                const int32_t *trow = p.pp.block_tables + static_cast<size_t>(b) * p.pp.W;
                mbar_arrive_expect_tx(k_full, Geo::kTileBytes);
#pragma unroll
                for (int i = 0; i < kKeys / kBlockTokens; ++i) {
                    const int blk = key_lo / kBlockTokens + i;
                    long long y = p.pp.num_blocks * p.pp.Hkv * kBlockTokens;  // past the tensor: zeros
                    if (blk < nblk) {
                        const int32_t phys = __ldg(trow + blk);
                        if (phys >= 0 && phys < p.pp.num_blocks)
                            y = (static_cast<long long>(phys) * p.pp.Hkv + kvh) * kBlockTokens;
                        else
                            flag(p.pp.err, PKV_DEV_ERR_BAD_BLOCK);
                    }
#pragma unroll
                    for (int hh = 0; hh < Geo::kHalves; ++hh)
                        tma_load_2d(smem_u32(smem) + hh * (128 * 128) + i * (kBlockTokens * 128), &tmk, hh * 64,
                                    static_cast<int>(y), k_full, policy);
                }
                int g = 0;
                for (; g < n; ++g) {
                    const int s = g % kQStages;
                    if (g >= kQStages &&
                        (!mbar_wait(q_empty(s), static_cast<uint32_t>((g / kQStages - 1) & 1), kWaitLimitNs) ||
                         *abort_flag)) {
                        flag(p.pp.err, PKV_DEV_ERR_TIMEOUT);
                        *abort_flag = 1;
                        break;
                    }
                    const int tok = sq.q0 + tok_lo + (i0 + g) * p.tile_tokens;
                    mbar_arrive_expect_tx(q_full(s), Geo::kHalves * rows * 128);
#pragma unroll
                    for (int hh = 0; hh < Geo::kHalves; ++hh)
                        tma_load_3d(smem_u32(smem + Geo::kQ + s * Geo::kTileBytes) + hh * (128 * 128), &tmq, hh * 64,
                                    kvh * G, tok, q_full(s), policy);
                }
                // on an abort, copies may still be landing: wait (bounded) for the last of each stage
                mbar_wait(k_full, 0, kWaitLimitNs);
                for (int i = max(g - kQStages, 0); i < g; ++i)
                    mbar_wait(q_full(i % kQStages), static_cast<uint32_t>((i / kQStages) & 1), kWaitLimitNs);
            }
        } else if (warp == kMmaWarp) {
            constexpr uint32_t kId = tc::idesc_bf16(kKeys, kCols, 0);
            bool ok = mbar_wait(k_full, 0, kWaitLimitNs);
            for (int g = 0; g < n && ok; ++g) {
                const int s = g % kQStages, x = g % kSBuffers;
                ok = mbar_wait(q_full(s), static_cast<uint32_t>((g / kQStages) & 1), kWaitLimitNs) && !*abort_flag;
                if (ok && g >= kSBuffers)
                    ok = mbar_wait(s_empty(x), static_cast<uint32_t>((g / kSBuffers - 1) & 1), kWaitLimitNs) &&
                         !*abort_flag;
                tc::fence_after();
                if (ok && lane == 0) {
                    const uint32_t kbase = smem_u32(smem), qbase = smem_u32(smem + Geo::kQ + s * Geo::kTileBytes);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int hh = k >> 2, kk = k & 3;
                        tc::mma_ss(tmem + kCols * x, tc::smem_desc(kbase + hh * (128 * 128) + kk * 32, 16, 1024),
                                   tc::smem_desc(qbase + hh * (128 * 128) + kk * 32, 16, 1024), kId, k > 0);
                    }
                    tc::commit(s_full(x));
                    tc::commit(q_empty(s));
                }
                __syncwarp();
            }
            if (!ok && lane == 0) {
                flag(p.pp.err, PKV_DEV_ERR_TIMEOUT);
                *abort_flag = 1;
            }
        } else {
            // ---------------- exponentials: thread t = TMEM lane t = key key_lo + t
            const int t = threadIdx.x;
            float *neg = reinterpret_cast<float *>(smem + Geo::kNeg);
            const float *lse = p.pp.lse + (static_cast<size_t>(kvh) * p.pp.num_tokens + sq.q0) * G;
            const uint32_t t_s = tmem + (static_cast<uint32_t>(warp * 32) << 16);
            const uint64_t scale2 = f2pack(p.pp.scale_log2, p.pp.scale_log2);
            const auto load_neg = [&](int g) {
                const int tok = tok_lo + (i0 + g) * p.tile_tokens;
                return t < min(p.tile_tokens, sq.nq - tok) * G ? -__ldcg(lse + static_cast<size_t>(tok) * G + t)
                                                               : -INFINITY;
            };
            float next = load_neg(0);
            bool ok = true;
            for (int g = 0; g < n; ++g) {
                const int x = g % kSBuffers;
                float *nb = neg + (g & 1) * kCols;
                nb[t] = next;
                if (g + 1 < n) next = load_neg(g + 1);
                asm volatile("bar.sync 1, 128;" ::: "memory");  // the exponential warps' buffer
                if (ok && (*abort_flag || !mbar_wait(s_full(x), static_cast<uint32_t>((g / kSBuffers) & 1), kWaitLimitNs)))
                    ok = false;
                // one vote for the four warps would cost a barrier: each warp leaves the loop by the
                // abort flag, but keeps meeting the others at the barrier above
                if (__any_sync(0xffffffffu, !ok)) {
                    ok = false;
                    if (lane == 0) {
                        flag(p.pp.err, PKV_DEV_ERR_TIMEOUT);
                        *abort_flag = 1;
                        mbar_arrive(s_empty(x));
                    }
                    continue;
                }
                tc::fence_after();
                const int tok = tok_lo + (i0 + g) * p.tile_tokens;
                const int count = min(p.tile_tokens, sq.nq - tok);
                // columns [c_lo, c_hi) are rows at or after this thread's key
                const int c_hi = count * G;
                const int before = key_lo + t - (sq.first_pos + tok);
                const int c_lo = before > 0 ? min(before, kCols) * G : 0;
                const bool diagonal = sq.first_pos + tok < key_lo + kKeys - 1;
                uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
                uint32_t sr[2][32];
                tc::ld32(t_s + kCols * x, sr[0]);
#pragma unroll
                for (int q = 0; q < kCols / 32; ++q) {
                    tc::wait_ld32(sr[q & 1]);
                    if (q + 1 < kCols / 32) tc::ld32(t_s + kCols * x + 32 * (q + 1), sr[(q + 1) & 1]);
                    const uint32_t *r = sr[q & 1];
                    // rows the tile does not have are left out by selection: theirs (zeros, or
                    // another sequence's queries) against a key that holds an infinity is NaN
                    const bool masked = diagonal || c_hi < 32 * (q + 1);
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const ulonglong2 nl = *reinterpret_cast<const ulonglong2 *>(nb + 32 * q + c);
                        float e[4];
                        f2unpack(ffma2(f2pack(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), scale2, nl.x), e[0], e[1]);
                        f2unpack(ffma2(f2pack(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), scale2, nl.y), e[2], e[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            e[i] = ex2_approx(e[i]);
                            if (masked) {
                                const int col = 32 * q + c + i;
                                e[i] = col >= c_lo && col < c_hi ? e[i] : 0.f;
                            }
                        }
                        acc[0] = fadd2(acc[0], f2pack(e[0], e[1]));
                        acc[1] = fadd2(acc[1], f2pack(e[2], e[3]));
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty(x));
                float a0, a1, a2, a3;
                f2unpack(acc[0], a0, a1);
                f2unpack(acc[1], a2, a3);
                total += (a0 + a1) + (a2 + a3);  // a tile's sum first: the total adds once a tile
            }
        }
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
        if (warp == kMmaWarp) tc::dealloc<kSBuffers * kCols>(tmem);
    }
    if (warp < kExpWarps) {
        const int pos = key_lo + threadIdx.x;
        if (pos < sq.ctx) {
            const size_t row = static_cast<size_t>(b) * p.pp.Hkv + kvh;
            if (p.splits > 1) {
                p.partial[(static_cast<size_t>(split) * p.pp.B * p.pp.Hkv + row) *
                              (static_cast<size_t>(p.pp.W) * kBlockTokens) + pos] = total;
            } else {
                const float in = p.sp.scores_in != nullptr && pos < sq.first_pos ? p.sp.scores_in[row * p.sp.stride + pos] : 0.f;
                p.sp.scores_out[row * p.sp.stride + pos] = in + total;
            }
        }
    }
}

constexpr int kJoinThreads = 256;

// The splits' sums, in order.
__global__ void __launch_bounds__(kJoinThreads) prefill_scores_join_kernel(const PrefillScoreParams p) {
    const int b = blockIdx.y / p.pp.Hkv;
    const size_t row = blockIdx.y;
    const int pos = blockIdx.x * kJoinThreads + threadIdx.x;
    ScoreSeq sq;
    if (!score_seq(p, b, sq) || pos >= sq.ctx) return;
    const size_t tokens = static_cast<size_t>(p.pp.W) * kBlockTokens;
    float x = p.sp.scores_in != nullptr && pos < sq.first_pos ? p.sp.scores_in[row * p.sp.stride + pos] : 0.f;
    float w = 0.f;
    for (int s = 0; s < p.splits; ++s)
        w += p.partial[(static_cast<size_t>(s) * p.pp.B * p.pp.Hkv + row) * tokens + pos];
    p.sp.scores_out[row * p.sp.stride + pos] = x + w;
}

template <int D>
cudaError_t launch_d(const CUtensorMap &tmk, const CUtensorMap &tmq, const PrefillScoreParams &p, cudaStream_t stream) {
    constexpr int kSmem = ScoreGeometry<D>::kSmemBytes;
    auto kern = prefill_scores_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const long long tokens = static_cast<long long>(p.pp.W) * kBlockTokens;
    // the first keys see the most queries: they go first
    const dim3 grid(static_cast<unsigned>(p.pp.B * p.pp.Hkv), static_cast<unsigned>((tokens + kKeys - 1) / kKeys),
                    static_cast<unsigned>(p.splits));
    kern<<<grid, kThreads, kSmem, stream>>>(tmk, tmq, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    const dim3 jgrid(static_cast<unsigned>((tokens + kJoinThreads - 1) / kJoinThreads),
                     static_cast<unsigned>(p.pp.B * p.pp.Hkv));
    prefill_scores_join_kernel<<<jgrid, kJoinThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

int prefill_score_splits(int B, int Hkv, int group, int W, int window, int max_query_len, int num_sms) {
    const long long units = static_cast<long long>(B) * Hkv * ((static_cast<long long>(W) * kBlockTokens + kKeys - 1) / kKeys);
    const long long tile_tokens = std::max(1, kCols / group);
    const long long tiles = (std::min(window, max_query_len) + tile_tokens - 1) / tile_tokens;
    // two waves of two CTAs per SM, at least two tiles each
    const long long want = (4LL * num_sms + units - 1) / std::max(1LL, units);
    return static_cast<int>(std::max(1LL, std::min({want, tiles / 2, 64LL})));
}

cudaError_t launch_prefill_scores(const CUtensorMap &tmk, const CUtensorMap &tmq, const PrefillScoreParams &p,
                                  int head_dim, cudaStream_t stream) {
    if (head_dim == 128) return launch_d<128>(tmk, tmq, p, stream);
    if (head_dim == 64) return launch_d<64>(tmk, tmq, p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
