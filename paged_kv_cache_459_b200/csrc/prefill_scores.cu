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
// of another.  The exponentials bound it: 128 x 128 of them take the
// special-function unit 1024 cycles, the tile's products 512.  Measured: 4 x
// 2048 tokens, 32 heads of 128, every query counted: 115 us (0.60 PFLOP/s).  Taken
// when it was 120: the two CTAs' warps take a tile pair in ~3100 cycles of the
// 2048 the unit needs (a warp alone 2300 for its 128 columns: the products'
// operand reads and the -lse reads share shared memory, 300 of them); eight
// exponential warps a CTA, a barrier a tile instead of the -lse warp, and a
// hand-ordered loop measured the same or slower (329, 350 and 329 us a call
// against 323).
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
constexpr int kExpWarps = 4;    // warp w: TMEM lanes 32 w .. 32 w + 31
constexpr int kProducerWarp = kExpWarps, kMmaWarp = kExpWarps + 1, kLseWarp = kExpWarps + 2;
constexpr int kThreads = (kExpWarps + 3) * 32;
constexpr int kQStages = 2;
constexpr int kSBuffers = 2;

template <int D>
struct ScoreGeometry {
    static constexpr int kHalves = D / 64;
    static constexpr int kTileBytes = kHalves * 128 * 128;  // K tile or Q tile: [half][row][128 B]
    static constexpr int kQ = kTileBytes;                   // + stage * kTileBytes
    static constexpr int kNeg = kQ + kQStages * kTileBytes;  // -lse of a tile's rows, beside each S buffer
    static constexpr int kBars = kNeg + kSBuffers * kCols * 4;
    static constexpr int kNumBars = 2 + 2 * kQStages + 2 * kSBuffers;
    static constexpr int kTmemSlot = kBars + kNumBars * 8;    // then the abort flag, a flag for each S buffer
    static constexpr int kSmemBytes = kTmemSlot + 8 + 4 * kSBuffers + 1024;
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

// One sequence's part in the scores.
struct ScoreSeq {
    int q0, nq, ctx, first_pos, first_tok;  // first_tok: first counted new token
};
// False for a sequence whose lengths do not fit.
__device__ __forceinline__ bool score_seq(const PrefillScoreParams &p, int b, ScoreSeq &s) {
    s.q0 = __ldg(p.pp.query_start + b);
    s.nq = max(__ldg(p.pp.query_start + b + 1) - s.q0, 0);
    s.ctx = __ldg(p.pp.seq_lens + b);
    s.first_pos = s.ctx - s.nq;
    s.first_tok = max(0, s.nq - p.window);
    return s.first_pos >= 0 && s.ctx <= p.pp.W * kBlockTokens && s.nq <= p.max_query_len &&
           (s.nq == 0 || (s.q0 >= 0 && s.q0 <= p.pp.num_tokens - s.nq));
}

// A unit: 128 keys of one (sequence, KV head), and a range of the query tiles
// that see some of them.
struct ScoreUnit {
    ScoreSeq sq;
    int b, kvh, split, key_lo;
    int tok;  // first new token of the range's first tile
    int n;    // tiles (0: nothing counted, the scores are still written)
};
// Units are numbered key tile first (the first keys see the most queries), then
// range, then (sequence, KV head).  False for keys past the sequence and for
// sequences whose lengths do not fit.
__device__ __forceinline__ bool score_unit(const PrefillScoreParams &p, int i, ScoreUnit &u) {
    const unsigned rows = static_cast<unsigned>(p.pp.B * p.pp.Hkv);
    unsigned rest = static_cast<unsigned>(i) / rows;
    const unsigned row = i - rest * rows;
    u.split = 0;
    if (p.splits > 1) {
        const unsigned tile = rest / static_cast<unsigned>(p.splits);
        u.split = static_cast<int>(rest - tile * p.splits);
        rest = tile;
    }
    u.key_lo = static_cast<int>(rest) * kKeys;
    u.b = static_cast<int>(row / static_cast<unsigned>(p.pp.Hkv));
    u.kvh = static_cast<int>(row) - u.b * p.pp.Hkv;
    if (!score_seq(p, u.b, u.sq) || u.key_lo >= u.sq.ctx) return false;
    const int tok_lo = max(u.sq.first_tok, u.key_lo - u.sq.first_pos);
    u.n = u.sq.nq > tok_lo ? static_cast<int>(static_cast<unsigned>(u.sq.nq - tok_lo + p.tile_tokens - 1) /
                                              static_cast<unsigned>(p.tile_tokens)) : 0;
    u.tok = tok_lo;
    if (p.splits > 1) {  // range `split` of the tiles; the first ones take the remainder
        const int base = u.n / p.splits, rem = u.n - base * p.splits;
        u.tok += (u.split * base + min(u.split, rem)) * p.tile_tokens;
        u.n = base + (u.split < rem);
    }
    return true;
}
// This CTA's next unit at or after round k (rounds of one unit a CTA, forwards
// and backwards in turn, so that heavy and light ones even out); its round or -1.
__device__ __forceinline__ int next_unit(const PrefillScoreParams &p, int k, ScoreUnit &u) {
    const int n = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    for (;; ++k) {
        const int i = k * n + ((k & 1) ? n - 1 - c : c);  // units + 2 n < 2^31
        if (i >= p.units) return -1;
        if (score_unit(p, i, u)) return k;
    }
}

// 2^x for x <= 0 on the FMA pipe, two at a time: x = n + f, n the nearest integer
// (by adding and taking away 1.5 * 2^23), 2^f by the degree-5 polynomial of
// least relative error on [-1/2, 1/2] (Remez exchange; 2.2e-7 in fp32), n added
// to the exponent.  Below 2^-125: 2^-125.
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t x2) {
    constexpr float kMagic = 12582912.f;
    float lo, hi;
    f2unpack(x2, lo, hi);
    x2 = f2pack(fmaxf(lo, -125.f), fmaxf(hi, -125.f));
    const uint64_t t2 = fadd2(x2, f2pack(kMagic, kMagic));
    const uint64_t n2 = fadd2(t2, f2pack(-kMagic, -kMagic));
    const uint64_t f2 = ffma2(n2, f2pack(-1.f, -1.f), x2);
    const auto c2 = [](float c) { return f2pack(c, c); };
    uint64_t r = ffma2(c2(0.0013276472454890609f), f2, c2(0.009675540961325169f));
    r = ffma2(r, f2, c2(0.05550713092088699f));
    r = ffma2(r, f2, c2(0.24022120237350464f));
    r = ffma2(r, f2, c2(0.6931469440460205f));
    r = ffma2(r, f2, c2(1.0000001192092896f));
    float tl, th, rl, rh;
    f2unpack(t2, tl, th);
    f2unpack(r, rl, rh);
    // the magic constant's own bits leave at the top
    return f2pack(__uint_as_float(__float_as_uint(rl) + (__float_as_uint(tl) << 23)),
                  __uint_as_float(__float_as_uint(rh) + (__float_as_uint(th) << 23)));
}

// The sum of 32 columns' weights 2^(scale s - lse).  MASKED: only columns
// [c_lo, c_hi); otherwise kPolyOf8 of every 8 pairs take the polynomial, so that
// the FMA pipe carries what the special-function unit, the bound, would not.
constexpr int kPolyOf8 = 1;  // a call of 4 x 2048 tokens: 331, 323, 323, 334 us with 0, 1, 2, 3
template <bool MASKED>
__device__ __forceinline__ void add_weights(const uint32_t *r, const float *nb, uint64_t scale2, int c_lo, int c_hi,
                                            uint64_t (&acc)[2]) {
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
        const ulonglong2 nl = *reinterpret_cast<const ulonglong2 *>(nb + c);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int col = c + 2 * h;
            const uint64_t x = ffma2(f2pack(__uint_as_float(r[col]), __uint_as_float(r[col + 1])), scale2, h ? nl.y : nl.x);
            const int pair = (col / 2) % 8;
            if (!MASKED && (pair * kPolyOf8) % 8 < kPolyOf8) {
                acc[h] = fadd2(acc[h], exp2_poly2(x));
            } else {
                float a, b;
                f2unpack(x, a, b);
                a = ex2_approx(a);
                b = ex2_approx(b);
                if (MASKED) {
                    a = col >= c_lo && col < c_hi ? a : 0.f;
                    b = col + 1 >= c_lo && col + 1 < c_hi ? b : 0.f;
                }
                acc[h] = fadd2(acc[h], f2pack(a, b));
            }
        }
    }
}

// Persistent, two CTAs per SM: every role walks the CTA's units; rings and
// phases run on across them, so a unit's first products are ready when the
// last one's exponentials end.
template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    prefill_scores_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmq,
                          const PrefillScoreParams p) {
    using Geo = ScoreGeometry<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.pp.group;
    const int rows = p.tile_tokens * G;  // rows a Q box fills

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t bar0 = smem_u32(smem + Geo::kBars);
    const uint32_t k_full = bar0, k_empty = bar0 + 8;
    const auto q_full = [&](int s) { return bar0 + 8 * (2 + s); };
    const auto q_empty = [&](int s) { return bar0 + 8 * (2 + kQStages + s); };
    const auto s_full = [&](int x) { return bar0 + 8 * (2 + 2 * kQStages + x); };
    const auto s_empty = [&](int x) { return bar0 + 8 * (2 + 2 * kQStages + kSBuffers + x); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Geo::kTmemSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Geo::kTmemSlot + 4);
    volatile int *odd_flag = abort_flag + 1;  // [kSBuffers]: a row of the tile has a sum that is not finite

    if (threadIdx.x == 0) {
        mbar_init(k_full, 1);
        mbar_init(k_empty, 1);
        for (int s = 0; s < kQStages; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
        }
        for (int x = 0; x < kSBuffers; ++x) {
            mbar_init(s_full(x), 2);  // its products and its rows' -lse
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
    // The join's CTAs (or the next call's) may take their places; they wait for
    // this grid.  Not before the allocation above: one of them, holding the right
    // to allocate while it waits, could keep this CTA from its columns for good.
    pdl_launch_dependents();

    if (warp == kProducerWarp) {
        if (lane == 0) {
            const uint64_t policy = l2_policy_evict_normal();
            int g = 0, nu = 0;  // Q tiles and K tiles loaded so far
            bool ok = true;
            const auto wait = [&](uint32_t bar, uint32_t parity) {
                if (ok && (!mbar_wait(bar, parity, kWaitLimitNs) || *abort_flag)) {
                    flag(p.pp.err, PKV_DEV_ERR_TIMEOUT);
                    *abort_flag = 1;
                    ok = false;
                }
                return ok;
            };
            ScoreUnit u;
            for (int k = next_unit(p, 0, u); k >= 0 && ok; k = next_unit(p, k + 1, u)) {
                if (u.n == 0) continue;
                for (int i = 0; i < u.n && ok; ++i, ++g) {
                    const int s = g % kQStages;
                    if (g >= kQStages && !wait(q_empty(s), static_cast<uint32_t>((g / kQStages - 1) & 1))) break;
                    mbar_arrive_expect_tx(q_full(s), Geo::kHalves * rows * 128);
#pragma unroll
                    for (int hh = 0; hh < Geo::kHalves; ++hh)
                        tma_load_3d(smem_u32(smem + Geo::kQ + s * Geo::kTileBytes) + hh * (128 * 128), &tmq, hh * 64,
                                    u.kvh * G, u.sq.q0 + u.tok + i * p.tile_tokens, q_full(s), policy);
                    if (i > 0) continue;
                    // the unit's keys, once the last unit's products have read theirs
                    if (nu > 0 && !wait(k_empty, static_cast<uint32_t>((nu - 1) & 1))) {
                        ++g;
                        break;
                    }
                    ++nu;
                    const int nblk = (u.sq.ctx + kBlockTokens - 1) / kBlockTokens;
                    const int32_t *trow = p.pp.block_tables + static_cast<size_t>(u.b) * p.pp.W;
                    mbar_arrive_expect_tx(k_full, Geo::kTileBytes);
#pragma unroll
                    for (int j = 0; j < kKeys / kBlockTokens; ++j) {
                        const int blk = u.key_lo / kBlockTokens + j;
                        long long y = p.pp.num_blocks * p.pp.Hkv * kBlockTokens;  // past the tensor: zeros
                        if (blk < nblk) {
                            const int32_t phys = __ldg(trow + blk);
                            if (phys >= 0 && phys < p.pp.num_blocks)
                                y = (static_cast<long long>(phys) * p.pp.Hkv + u.kvh) * kBlockTokens;
                            else
                                flag(p.pp.err, PKV_DEV_ERR_BAD_BLOCK);
                        }
#pragma unroll
                        for (int hh = 0; hh < Geo::kHalves; ++hh)
                            tma_load_2d(smem_u32(smem) + hh * (128 * 128) + j * (kBlockTokens * 128), &tmk, hh * 64,
                                        static_cast<int>(y), k_full, policy);
                    }
                }
            }
            // on an abort, copies may still be landing: wait (bounded) for the last of each stage
            if (nu > 0) mbar_wait(k_full, static_cast<uint32_t>((nu - 1) & 1), kWaitLimitNs);
            for (int i = max(g - kQStages, 0); i < g; ++i)
                mbar_wait(q_full(i % kQStages), static_cast<uint32_t>((i / kQStages) & 1), kWaitLimitNs);
            // sequences whose lengths do not fit: flagged once each
            for (int b = blockIdx.x; b < p.pp.B; b += gridDim.x) {
                ScoreSeq sq;
                if (!score_seq(p, b, sq)) flag(p.pp.err, PKV_DEV_ERR_BAD_LEN);
            }
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t kId = tc::idesc_bf16(kKeys, kCols, 0);
        // a lane that gives up walks on with the others, as in the attention kernel
        bool ok = true;
        const auto wait = [&](uint32_t bar, uint32_t parity) {
            if (ok && (!mbar_wait(bar, parity, kWaitLimitNs) || *abort_flag)) {
                ok = false;
                flag(p.pp.err, PKV_DEV_ERR_TIMEOUT);
                *abort_flag = 1;
            }
        };
        int g = 0, nu = 0;
        ScoreUnit u;
        for (int k = next_unit(p, 0, u); k >= 0; k = next_unit(p, k + 1, u)) {
            if (u.n == 0) continue;
            wait(k_full, static_cast<uint32_t>(nu & 1));
            for (int i = 0; i < u.n; ++i, ++g) {
                const int s = g % kQStages, x = g % kSBuffers;
                wait(q_full(s), static_cast<uint32_t>((g / kQStages) & 1));
                if (g >= kSBuffers) wait(s_empty(x), static_cast<uint32_t>((g / kSBuffers - 1) & 1));
                tc::fence_after();
                if (ok && lane == 0) {
                    const uint32_t kbase = smem_u32(smem), qbase = smem_u32(smem + Geo::kQ + s * Geo::kTileBytes);
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        const int hh = d >> 2, kk = d & 3;
                        tc::mma_ss(tmem + kCols * x, tc::smem_desc(kbase + hh * (128 * 128) + kk * 32, 16, 1024),
                                   tc::smem_desc(qbase + hh * (128 * 128) + kk * 32, 16, 1024), kId, d > 0);
                    }
                    tc::commit(s_full(x));
                    tc::commit(q_empty(s));
                    if (i + 1 == u.n) tc::commit(k_empty);
                }
                __syncwarp();
            }
            ++nu;
        }
    } else if (warp == kLseWarp) {
        // -lse of each tile's rows (-inf for a row the tile does not have), four
        // columns a lane, the next tile's on their way while this one waits for
        // its buffer: the exponential warps meet only at mbarriers.
        float *neg = reinterpret_cast<float *>(smem + Geo::kNeg);
        const auto load = [&](const ScoreUnit &v, int i, float (&x)[4]) {
            const int tok = v.tok + i * p.tile_tokens;
            const int cols = min(p.tile_tokens, v.sq.nq - tok) * G;
            const float *row = p.pp.lse + (static_cast<size_t>(v.kvh) * p.pp.num_tokens + v.sq.q0 + tok) * G;
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = 4 * lane + e;
                x[e] = c < cols ? -__ldcg(row + c) : -INFINITY;
                odd = odd || (c < cols && !(fabsf(x[e]) < INFINITY));
            }
            return odd;
        };
        bool ok = true;
        int g = 0;
        ScoreUnit u, nx;
        float x4[4];
        bool odd = false;
        int k = next_unit(p, 0, u);
        while (k >= 0 && u.n == 0) k = next_unit(p, k + 1, u);
        if (k >= 0) odd = load(u, 0, x4);
        while (k >= 0 && ok) {
            int kn = next_unit(p, k + 1, nx);
            while (kn >= 0 && nx.n == 0) kn = next_unit(p, kn + 1, nx);
            for (int i = 0; i < u.n; ++i, ++g) {
                const int x = g % kSBuffers;
                if (g >= kSBuffers &&
                    !mbar_wait_warp(s_empty(x), static_cast<uint32_t>((g / kSBuffers - 1) & 1), kWaitLimitNs, abort_flag)) {
                    ok = false;
                    break;
                }
                *reinterpret_cast<float4 *>(neg + x * kCols + 4 * lane) = make_float4(x4[0], x4[1], x4[2], x4[3]);
                odd = __any_sync(0xffffffffu, odd);
                if (lane == 0) odd_flag[x] = odd;
                __syncwarp();
                if (lane == 0) mbar_arrive(s_full(x));
                if (i + 1 < u.n)
                    odd = load(u, i + 1, x4);
                else if (kn >= 0)
                    odd = load(nx, 0, x4);
            }
            u = nx;
            k = kn;
        }
        if (!ok && lane == 0) {
            flag(p.pp.err, PKV_DEV_ERR_TIMEOUT);
            *abort_flag = 1;
        }
    } else {
        // ---------------- exponentials: thread t = TMEM lane t = key key_lo + t
        const int t = threadIdx.x;
        const float *neg = reinterpret_cast<const float *>(smem + Geo::kNeg);
        const uint32_t t_s = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const uint64_t scale2 = f2pack(p.pp.scale_log2, p.pp.scale_log2);
        bool ok = true;
        int g = 0;
        ScoreUnit u, nx;
        int k = next_unit(p, 0, u);
        while (k >= 0 && ok) {
            const int kn = next_unit(p, k + 1, nx);
            float total = 0.f;
            for (int i = 0; i < u.n; ++i, ++g) {
                const int x = g % kSBuffers;
                ok = mbar_wait_warp(s_full(x), static_cast<uint32_t>((g / kSBuffers) & 1), kWaitLimitNs);
                if (!ok) break;
                tc::fence_after();
                uint32_t sr[2][32];
                const uint32_t ts = t_s + kCols * x;
                tc::ld32(ts, sr[0]);
                // columns [c_lo, c_hi) are rows at or after this thread's key
                const int tok = u.tok + i * p.tile_tokens;
                const int c_hi = min(p.tile_tokens, u.sq.nq - tok) * G;
                const bool diagonal = u.sq.first_pos + tok < u.key_lo + kKeys - 1;
                const int before = u.key_lo + t - (u.sq.first_pos + tok);
                const int c_lo = before > 0 ? min(before, kCols) * G : 0;
                // Rows the tile does not have are left out by selection (theirs -- zeros, or another
                // sequence's queries -- against a key that holds an infinity are NaN), and where a row's own
                // sum is not finite every weight goes through the special-function unit, which keeps
                // infinities and NaN as they are.
                const bool odd = odd_flag[x];
                uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
                const auto chunk = [&](const uint32_t *r, int c0) {
                    // no row of the chunk sees a key of the warp / every one sees every key
                    if (diagonal && __all_sync(0xffffffffu, c_lo >= c0 + 32)) return;
                    const bool some = odd || c_hi < c0 + 32 || (diagonal && !__all_sync(0xffffffffu, c_lo <= c0));
                    const float *nb = neg + x * kCols + c0;
                    if (some)
                        add_weights<true>(r, nb, scale2, c_lo - c0, c_hi - c0, acc);
                    else
                        add_weights<false>(r, nb, scale2, 0, 32, acc);
                };
#pragma unroll 1  // two chunks' code, not four
                for (int q = 0; q < kCols; q += 64) {
                    tc::wait_ld32(sr[0]);
                    tc::ld32(ts + q + 32, sr[1]);
                    chunk(sr[0], q);
                    tc::wait_ld32(sr[1]);
                    if (q + 64 < kCols) tc::ld32(ts + q + 64, sr[0]);
                    chunk(sr[1], q + 32);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty(x));
                float a0, a1, a2, a3;
                f2unpack(acc[0], a0, a1);
                f2unpack(acc[1], a2, a3);
                total += (a0 + a1) + (a2 + a3);  // a tile's sum first: the total adds once a tile
            }
            if (!ok) break;
            const int pos = u.key_lo + t;
            if (pos < u.sq.ctx) {
                const size_t row = static_cast<size_t>(u.b) * p.pp.Hkv + u.kvh;
                if (p.splits > 1) {
                    p.partial[(static_cast<size_t>(u.split) * p.pp.B * p.pp.Hkv + row) *
                                  (static_cast<size_t>(p.pp.W) * kBlockTokens) + pos] = total;
                } else {
                    const float in = p.sp.scores_in != nullptr && pos < u.sq.first_pos ? p.sp.scores_in[row * p.sp.stride + pos] : 0.f;
                    p.sp.scores_out[row * p.sp.stride + pos] = in + total;
                }
            }
            u = nx;
            k = kn;
        }
        if (!ok && lane == 0) {
            flag(p.pp.err, PKV_DEV_ERR_TIMEOUT);
            *abort_flag = 1;
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kMmaWarp) tc::dealloc<kSBuffers * kCols>(tmem);
}

constexpr int kJoinThreads = 256;

// The splits' sums, in order.
__global__ void __launch_bounds__(kJoinThreads) prefill_scores_join_kernel(const PrefillScoreParams p) {
    pdl_launch_dependents();
    const int b = blockIdx.y / p.pp.Hkv;
    const size_t row = blockIdx.y;
    const int pos = blockIdx.x * kJoinThreads + threadIdx.x;
    pdl_wait_primary();
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
cudaError_t launch_d(const CUtensorMap &tmk, const CUtensorMap &tmq, PrefillScoreParams p, int num_sms,
                     cudaStream_t stream) {
    constexpr int kSmem = ScoreGeometry<D>::kSmemBytes;
    auto kern = prefill_scores_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const long long tokens = static_cast<long long>(p.pp.W) * kBlockTokens;
    const long long units = (tokens + kKeys - 1) / kKeys * p.splits * p.pp.B * p.pp.Hkv;
    if (units > INT32_MAX - 8LL * num_sms) return cudaErrorInvalidValue;
    p.units = static_cast<int>(units);
    const unsigned grid = static_cast<unsigned>(std::min<long long>(units, 2LL * num_sms));
    kern<<<grid, kThreads, kSmem, stream>>>(tmk, tmq, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    const dim3 jgrid(static_cast<unsigned>((tokens + kJoinThreads - 1) / kJoinThreads),
                     static_cast<unsigned>(p.pp.B * p.pp.Hkv));
    return launch_dependent(prefill_scores_join_kernel, jgrid, dim3(kJoinThreads), stream, p);
}

}  // namespace

int prefill_score_splits(int B, int Hkv, int group, int W, int window, int max_query_len, int num_sms) {
    const long long units = static_cast<long long>(B) * Hkv * ((static_cast<long long>(W) * kBlockTokens + kKeys - 1) / kKeys);
    const long long tile_tokens = std::max(1, kCols / group);
    const long long tiles = (std::min(window, max_query_len) + tile_tokens - 1) / tile_tokens;
    // two waves of two CTAs per SM, a tile each at least (short prompts: 20 us a call, 22 with two tiles, 25 with eight)
    const long long want = (4LL * num_sms + units - 1) / std::max(1LL, units);
    return static_cast<int>(std::max(1LL, std::min({want, tiles, 64LL})));
}

cudaError_t launch_prefill_scores(const CUtensorMap &tmk, const CUtensorMap &tmq, const PrefillScoreParams &p,
                                  int head_dim, int num_sms, cudaStream_t stream) {
    if (head_dim == 128) return launch_d<128>(tmk, tmq, p, num_sms, stream);
    if (head_dim == 64) return launch_d<64>(tmk, tmq, p, num_sms, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
