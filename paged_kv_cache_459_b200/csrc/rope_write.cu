// Rotary positions fused with the paged cache write.
//
// Pair i of a head's first `rot` elements -- (i, i + rot/2), or (2i, 2i + 1)
// when interleaved -- turns by the angle of position P = positions[axis(i)][t]:
//   x1' = x1 cos - x2 sin,  x2' = x2 cos + x1 sin,   cos, sin = cos_sin[P][i], [P][rot/2 + i]
// in fp32, rounded to bf16 once.  q rows go to q_out, k rows to the token's
// cache slot, v rows are copied to theirs.
//
// Every byte moves once, so the kernel is bound by HBM for prompts and by the
// launch for decode steps.  A lane owns one item of a row -- two 16-byte
// vectors that hold 8 whole pairs -- in every row its warp takes, so the
// token's 8 cosines and 8 sines are read once and stay in registers while the
// warp walks the token's q, k and v rows, kBatch rows' loads in flight.  Measured,
// calls back to back: 7411 tokens, 28/4 heads, 3 axes, 24.7 us (5.7 TB/s; 25.5 with
// kBatch 2, 25.7 with 4, 30.3 with a warp for every kBatch rows instead of a whole
// token); 32768 tokens, 32/8 heads of 64, half rotated, 64.0 us (6.36 TB/s; 64.0,
// 65.1 and 63.6); 64 tokens 2.7 us.
#include "decode_common.cuh"

namespace pkv {

namespace {

using namespace dev;

constexpr int kRopeThreads = 128;
constexpr int kBatch = 3;  // rows a lane has in flight

// 8 pairs: a holds the first elements, b the second (half-split), or the 16
// elements in order (interleaved).
template <bool INTER>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const float (&c)[8], const float (&s)[8]) {
    uint32_t *pa = reinterpret_cast<uint32_t *>(&a), *pb = reinterpret_cast<uint32_t *>(&b);
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t &w = i < 4 ? pa[i] : pb[i - 4];
            const float x1 = bf16lo(w), x2 = bf16hi(w);
            w = pack_bf16x2(x1 * c[i] - x2 * s[i], x2 * c[i] + x1 * s[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x1 = bf16lo(pa[i]), x2 = bf16lo(pb[i]), y1 = bf16hi(pa[i]), y2 = bf16hi(pb[i]);
            const float c0 = c[2 * i], s0 = s[2 * i], c1 = c[2 * i + 1], s1 = s[2 * i + 1];
            pa[i] = pack_bf16x2(x1 * c0 - x2 * s0, y1 * c1 - y2 * s1);
            pb[i] = pack_bf16x2(x2 * c0 + x1 * s0, y2 * c1 + y1 * s1);
        }
    }
}

// One warp per (token, range of `rows_per_unit` of its Hq + 2 Hkv rows).
template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kv_write_kernel(const RopeParams p, int rows_per_unit, int units_per_token) {
    constexpr int kItems = D / 16;         // items (lanes) per row
    constexpr int kRows = 32 / kItems;     // rows of one pass of the warp
    pdl_launch_dependents();
    const long long unit = (static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x) / 32;
    const int lane = threadIdx.x & 31;
    const int item = lane % kItems;
    const long long t = unit / units_per_token;
    pdl_wait_primary();
    if (t >= p.T) return;
    const int total = p.Hq + 2 * p.Hkv;
    const int row0 = static_cast<int>(unit % units_per_token) * rows_per_unit;
    const int row1 = min(total, row0 + rows_per_unit);

    // element offsets of the lane's two vectors
    const int half = p.rot / 2;
    const bool turned = item < p.rot / 16;
    int ea, eb;
    if (INTER || !turned) {
        ea = item * 16;
        eb = ea + 8;
    } else {
        ea = item * 8;
        eb = ea + half;
    }

    uint4 a[kBatch], b[kBatch];
    const auto load = [&](int base) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int r = base + j * kRows + lane / kItems;
            if (r < row1) {
                const __nv_bfloat16 *src =
                    r < p.Hq ? p.q + t * p.q_stride + r * D
                    : r < p.Hq + p.Hkv ? p.k + t * p.k_stride + (r - p.Hq) * D
                                       : p.v + t * p.v_stride + (r - p.Hq - p.Hkv) * D;
                a[j] = *reinterpret_cast<const uint4 *>(src + ea);
                b[j] = *reinterpret_cast<const uint4 *>(src + eb);
            }
        }
    };
    // the first rows are on their way while slot, position and then the table's row are read
    load(row0);

    const long long slot = p.slots[t];
    long long pos[8];
    bool ok = true;
    if (p.axes == 1) {
        const long long q = p.positions[t];
        ok = q >= 0 && q < p.max_positions;
#pragma unroll
        for (int i = 0; i < 8; ++i) pos[i] = q;
    } else {
        long long ax[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            ax[a] = a < p.axes ? p.positions[static_cast<long long>(a) * p.T + t] : 0;
            ok = ok && ax[a] >= 0 && ax[a] < p.max_positions;
        }
        const uint32_t bits = turned ? (p.axis_bits[item >> 1] >> (16 * (item & 1))) & 0xFFFFu : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = (bits >> (2 * i)) & 3u;
            pos[i] = a == 0 ? ax[0] : a == 1 ? ax[1] : a == 2 ? ax[2] : ax[3];
        }
    }
    if (!ok) {  // warp-uniform: the whole token is left out
        if (lane == 0 && row0 == 0) flag(p.err, PKV_DEV_ERR_BAD_POS);
        return;
    }
    const bool in_pool = slot >= 0 && slot < p.num_blocks * kBlockTokens;
    if (slot >= 0 && !in_pool && lane == 0 && row0 == 0) flag(p.err, PKV_DEV_ERR_BAD_SLOT);
    const long long blk = in_pool ? slot / kBlockTokens : 0;
    const int off = in_pool ? static_cast<int>(slot % kBlockTokens) : 0;

    float c[8], s[8];
    if (turned) {
        const int i0 = item * 8;
        bool same = true;
#pragma unroll
        for (int i = 1; i < 8; ++i) same = same && pos[i] == pos[0];
        if (same) {
            const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + pos[0] * p.rot + i0);
            const float4 *srow = reinterpret_cast<const float4 *>(p.cos_sin + pos[0] * p.rot + half + i0);
            *reinterpret_cast<float4 *>(c) = row[0];
            *reinterpret_cast<float4 *>(c + 4) = row[1];
            *reinterpret_cast<float4 *>(s) = srow[0];
            *reinterpret_cast<float4 *>(s + 4) = srow[1];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = p.cos_sin[pos[i] * p.rot + i0 + i];
                s[i] = p.cos_sin[pos[i] * p.rot + half + i0 + i];
            }
        }
    }

    for (int base = row0; base < row1; base += kRows * kBatch) {
        if (base > row0) load(base);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int r = base + j * kRows + lane / kItems;
            if (r >= row1) continue;
            __nv_bfloat16 *dst;
            if (r < p.Hq) {
                dst = p.q_out + t * p.q_out_stride + r * D;
            } else {
                if (!in_pool) continue;
                const bool is_v = r >= p.Hq + p.Hkv;
                const int h = r - p.Hq - (is_v ? p.Hkv : 0);
                dst = (is_v ? p.v_cache : p.k_cache) + ((blk * p.Hkv + h) * kBlockTokens + off) * D;
            }
            if (turned && r < p.Hq + p.Hkv) rotate<INTER>(a[j], b[j], c, s);
            *reinterpret_cast<uint4 *>(dst + ea) = a[j];
            *reinterpret_cast<uint4 *>(dst + eb) = b[j];
        }
    }
}

template <int D, bool INTER>
cudaError_t launch_rope(const RopeParams &p, int num_sms, cudaStream_t stream) {
    constexpr int kPass = 32 / (D / 16) * kBatch;  // rows of one batch of the warp
    const int total = p.Hq + 2 * p.Hkv;
    // as many batches per warp as leave 16 warps for every SM
    int batches = (total + kPass - 1) / kPass;
    while (batches > 1 && static_cast<long long>(p.T) * ((total + kPass * batches - 1) / (kPass * batches)) < 16LL * num_sms)
        --batches;
    const int rows_per_unit = kPass * batches;
    const int units = (total + rows_per_unit - 1) / rows_per_unit;
    const long long warps = static_cast<long long>(p.T) * units;
    const long long ctas = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    return launch_dependent(rope_kv_write_kernel<D, INTER>, dim3(static_cast<unsigned>(ctas)), dim3(kRopeThreads),
                            stream, p, rows_per_unit, units);
}

}  // namespace

cudaError_t launch_rope_kv_write(const RopeParams &p, int head_dim, bool interleaved, int num_sms,
                                 cudaStream_t stream) {
    if (head_dim == 128)
        return interleaved ? launch_rope<128, true>(p, num_sms, stream) : launch_rope<128, false>(p, num_sms, stream);
    if (head_dim == 64)
        return interleaved ? launch_rope<64, true>(p, num_sms, stream) : launch_rope<64, false>(p, num_sms, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
