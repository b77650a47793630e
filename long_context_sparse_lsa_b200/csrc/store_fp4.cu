// store_fp4.cu — new K/V rows into the 4-bit cache, for any number of new
// tokens of packed sequences (one per sequence in a decode step, a whole
// prompt, a batch of prompts of different lengths).
//
// For each group of 16 channels x of a row and the layer's scale S (a power
// of two):
//   s    = E4M3(max|x| / (6 S)),  to nearest, ties to even, at most 448
//   code = E2M1(x / (s S)),       to nearest, ties to even, at most 6
// s == 0 stores codes 0; a group with a number that is not finite stores the
// scale NaN (0x7f) and codes 0, and sets LSA_DEV_BAD_VALUE.
//
// Exact rounding in fp32. A power of two changes no significant bit, so S = 1
// below. x has at most 8 significant bits and s at most 4. A border t between
// two codes is a multiple of 1/4 of 3 bits: t and x / s are equal or at least
// t * 2^-8 >= 2^-10 apart. The quotient by a reciprocal (off by a few 2^-24)
// rounded to a multiple of 2^-13 is therefore on the right side of every border,
// and exactly on it in a tie. For the scale, a border b of E4M3 has 5 bits and
// 6 b has 7: it and max|x| are equal or more than 2^-8 of themselves apart, so
// max|x| * (1/6) rounded to 12 significant bits is on b's right side, and on b
// in a tie.
//
// Bound: HBM bytes (2 read, 9/16 written per number, 2 more with the rounded
// rows: 306 MB for 65536 tokens of 4 heads, 49 us); with a few rows, the latency
// of the dependent loads. With an IEEE division and reciprocal per group, a
// 64-bit division per thread and seven operations per number the instructions
// bound it (85% of the issue slots, 56 us). A thread per group or two: 32 bytes in, 8
// code bytes and 1 scale byte out, consecutive threads on consecutive groups,
// so that every access of a warp is a run.
#include "fp4.cuh"
#include "internal.h"

namespace lsa {
namespace {

constexpr int kStThreads = 256;

struct Groups16 {
    uint4 a, b;  // 16 bf16
};

// One group: codes (8 bytes), scale byte, and the values they stand for.
struct GroupFp4 {
    uint32_t code[2];
    uint32_t scale;
    uint32_t value[8];  // 16 bf16
    bool bad;
};

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

template <bool VALUES>
__device__ __forceinline__ void quantise(const Groups16& in, float S, float inv_S, GroupFp4& out) {
    const uint32_t w[8] = {in.a.x, in.a.y, in.a.z, in.a.w, in.b.x, in.b.y, in.b.z, in.b.w};
    // the largest magnitude: bf16 magnitudes order as their 15 bits do, NaN above infinity
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    out.bad = top >= 0x7f80u;
    const float sixth = fminf(__uint_as_float(top << 16) * (inv_S * (1.f / 6.f)), 1024.f);
    const float up = __fmul_rn(sixth, 4097.f);  // to 12 significant bits (not to be fused into one operation)
    const float want = __fsub_rn(up, __fsub_rn(up, sixth));
    const uint32_t byte = (uint32_t)__nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
    out.scale = out.bad ? kE4m3NaN : byte;
    const float s = e4m3_to_f32(out.scale);
    const bool live = !out.bad && byte != 0;
    float f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(s));
    f = live ? f * inv_S : 0.f;
    // 1536 = 1.5 * 2^10: adding it rounds to a multiple of 2^-13 (numbers it does not
    // fit are above 6 on either side of the rounding)
    const f32x2 f2 = pair(f, f), big = pair(1536.f, 1536.f), neg_big = pair(-1536.f, -1536.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float r[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = bf16_lo(w[4 * h + i]), hi = bf16_hi(w[4 * h + i]);
            float t0, t1;
            unpair(add2(fma2(pair(lo, hi), f2, big), neg_big), t0, t1);
            r[2 * i] = copysignf(t0, lo);
            r[2 * i + 1] = copysignf(t1, hi);
        }
        out.code[h] = live ? f32_to_e2m1x8(r) : 0u;
    }
    if (VALUES) {
        const float sS = s * S;  // exact; NaN for a group that is not finite
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t p[4];
            e2m1x8_to_f16(out.code[h], p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
                float v0, v1;
                unpair(mul2(pair(v.x, v.y), pair(sS, sS)), v0, v1);
                out.value[4 * h + i] = pack_bf16(v0, v1);
            }
        }
    }
}

// grid: (runs of PER * kStThreads groups, layers * 2): K of layer g at y = 2 g, V
// at 2 g + 1. A thread takes PER groups, kStThreads apart, all asked for at once.
template <bool VALUES, int PER>
__global__ void __launch_bounds__(kStThreads) store_fp4_kernel(const __grid_constant__ StoreFp4Args a) {
    constexpr int kPairs = PER * kStThreads / kFp4Groups;  // (row, head) pairs of a CTA
    __shared__ int64_t s_dst[kPairs + 2];
    const int tid = threadIdx.x;
    const int layer = blockIdx.y >> 1, is_v = blockIdx.y & 1;
    const int per_row = a.H_kv * kFp4Groups;
    // (the number of pairs fits 32 bits, as n_rows * H_kv does)
    const uint32_t pair0 = blockIdx.x * (uint32_t)kPairs, H = (uint32_t)a.H_kv;
    const uint32_t first = pair0 / H;
    const int row0 = (int)first;
    int row[PER], in_row[PER];
    Groups16 x[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const uint32_t head = pair0 - first * H + (uint32_t)(u * (kStThreads / kFp4Groups) + tid / kFp4Groups);
        row[u] = row0 + (int)(head / H);
        in_row[u] = (int)(head % H) * kFp4Groups + tid % kFp4Groups;
    }
    pdl_enter();
    const uint16_t* src = is_v ? a.v_new[layer] : a.k_new[layer];
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        x[u] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (row[u] < a.n_rows) {
            const uint16_t* p = src + (int64_t)row[u] * stride + in_row[u] * kFp4Group;
            x[u].a = *reinterpret_cast<const uint4*>(p);
            x[u].b = *reinterpret_cast<const uint4*>(p + 8);
        }
    }
    // cache rows of the CTA's tokens
    if (tid < kWarp) {
        const int last = min(a.n_rows - 1, (int)((pair0 + kPairs - 1) / H));
        int seq = find_last(a.n_seq, [&](int b) { return a.row_offset[b] <= row0; });
        for (int i = tid; i <= last - row0; i += kWarp) {
            const int r = row0 + i;
            while (seq + 1 < a.n_seq && a.row_offset[seq + 1] <= r) ++seq;
            const int lo = a.row_offset[seq], hi = a.row_offset[seq + 1];
            const int len = a.seq_lens[seq];
            const int64_t off = a.kv_offset[seq];
            int64_t dst = -1;
            if (r >= lo && r < hi) {
                if (hi <= a.n_rows && lo >= 0 && hi - lo <= len && len <= a.max_len && off >= 0 &&
                    off <= a.total_tokens - len)
                    dst = off + len - (hi - r);
                else
                    flag(a.dev_status, LSA_DEV_BAD_LENGTH);
            }
            s_dst[i] = dst;
        }
    }
    if (blockIdx.x + blockIdx.y == 0 && tid == kWarp && rows_outside(a.row_offset, a.n_seq, a.n_rows))
        flag(a.dev_status, LSA_DEV_BAD_LENGTH);
    const float S = is_v ? a.v_scale[layer] : a.k_scale[layer];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        if (row[u] >= a.n_rows) return;
        const int64_t dst = s_dst[row[u] - row0];
        if (dst < 0) continue;
        GroupFp4 q;
        quantise<VALUES>(x[u], S, 1.f / S, q);
        if (q.bad) flag(a.dev_status, LSA_DEV_BAD_VALUE);
        const int64_t to = dst * per_row + in_row[u];
        *reinterpret_cast<uint2*>((is_v ? a.v[layer] : a.k[layer]) + to * 8) = make_uint2(q.code[0], q.code[1]);
        (is_v ? a.v_group[layer] : a.k_group[layer])[to] = (uint8_t)q.scale;
        if (VALUES) {
            uint16_t* out = is_v ? a.v_round[layer] : a.k_round[layer];
            if (out != nullptr) {
                uint4* p = reinterpret_cast<uint4*>(out + ((int64_t)row[u] * per_row + in_row[u]) * kFp4Group);
                p[0] = make_uint4(q.value[0], q.value[1], q.value[2], q.value[3]);
                p[1] = make_uint4(q.value[4], q.value[5], q.value[6], q.value[7]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_store_fp4(const StoreFp4Args& a, cudaStream_t stream) {
    const int64_t groups = (int64_t)a.n_rows * a.H_kv * kFp4Groups;
    // Two groups a thread where one each would be more than two rounds of the eight
    // CTAs that an SM holds: half the searches and more bytes in flight (65536
    // tokens, 4 heads 48.7 against 52.2 us, 16000 tokens 15.6 and 16.2; 16 tokens
    // 3.8 and 3.1).
    const int64_t ctas = (groups + kStThreads - 1) / kStThreads * 2 * a.layers;
    const bool two = ctas > 16 * (int64_t)device_sm_count();
    const int per = two ? 2 : 1;
    auto kern = a.values ? (two ? store_fp4_kernel<true, 2> : store_fp4_kernel<true, 1>)
                         : (two ? store_fp4_kernel<false, 2> : store_fp4_kernel<false, 1>);
    const dim3 grid((unsigned)((groups + per * kStThreads - 1) / (per * kStThreads)), (unsigned)(2 * a.layers));
    return launch_pdl(kern, grid, dim3(kStThreads), 0, stream, 0, a);
}

}  // namespace lsa
