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
// Exact rounding in fp32. x / S is exact (a power of two). x has at most 8
// significant bits and s at most 4, so a border t between two codes (a
// multiple of 1/4, 3 bits) and x / (s S) are either equal or at least
// t * 2^-8 >= 2^-10 apart: the quotient taken by a reciprocal (off by a few
// 2^-24) and then rounded to a multiple of 2^-13 is on the right side of
// every border and exactly on it in a tie. The same holds for max|x| / (6 S)
// and E4M3's borders (5 significant bits), where one IEEE division per group
// does.
//
// Bound: HBM bytes (2 read, 9/16 written per number, 2 more with the rounded
// rows); with a few rows, the latency of the dependent loads. One thread per
// group: 32 bytes in, 8 code bytes and 1 scale byte out, consecutive threads
// on consecutive groups, so that every access of a warp is a run.
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
    const float want = __fdiv_rn(__uint_as_float(top << 16) * inv_S, 6.f);
    const uint32_t byte = (uint32_t)__nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
    out.scale = out.bad ? kE4m3NaN : byte;
    const float s = e4m3_to_f32(out.scale);
    const bool live = !out.bad && byte != 0;
    const float f = live ? __frcp_rn(s) : 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float r[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = w[4 * h + i];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float v = e ? bf16_hi(x) : bf16_lo(x);
                // 1536 = 1.5 * 2^10: adding it rounds to a multiple of 2^-13
                const float t = (fminf(fabsf(v) * inv_S * f, 8.f) + 1536.f) - 1536.f;
                r[2 * i + e] = copysignf(t, v);
            }
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
                out.value[4 * h + i] = pack_bf16(v.x * sS, v.y * sS);
            }
        }
    }
}

// grid: (runs of kStThreads groups, layers * 2): K of layer g at y = 2 g, V at 2 g + 1
template <bool VALUES>
__global__ void __launch_bounds__(kStThreads) store_fp4_kernel(const __grid_constant__ StoreFp4Args a) {
    __shared__ int64_t s_dst[kStThreads / kFp4Groups + 2];
    const int tid = threadIdx.x;
    const int layer = blockIdx.y >> 1, is_v = blockIdx.y & 1;
    const int per_row = a.H_kv * kFp4Groups;
    const int64_t g0 = (int64_t)blockIdx.x * kStThreads;
    const int64_t idx = g0 + tid;
    const int row0 = (int)(g0 / per_row);
    const int row = (int)(idx / per_row);
    const int in_row = (int)(idx - (int64_t)row * per_row);
    const bool live = row < a.n_rows;
    pdl_enter();
    Groups16 x = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (live) {
        const uint16_t* src = (is_v ? a.v_new[layer] : a.k_new[layer]) + (int64_t)row * (is_v ? a.v_stride : a.k_stride) +
                              in_row * kFp4Group;
        x.a = *reinterpret_cast<const uint4*>(src);
        x.b = *reinterpret_cast<const uint4*>(src + 8);
    }
    // cache rows of the CTA's tokens
    if (tid < kWarp) {
        const int last = min(a.n_rows - 1, (int)((g0 + kStThreads - 1) / per_row));
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
                    off + len <= a.total_tokens)
                    dst = off + len - (hi - r);
                else
                    flag(a.dev_status, LSA_DEV_BAD_LENGTH);
            }
            s_dst[i] = dst;
        }
    }
    GroupFp4 q;
    const float S = is_v ? a.v_scale[layer] : a.k_scale[layer];
    quantise<VALUES>(x, S, 1.f / S, q);
    __syncthreads();
    if (!live) return;
    const int64_t dst = s_dst[row - row0];
    if (dst < 0) return;
    if (q.bad) flag(a.dev_status, LSA_DEV_BAD_VALUE);
    const int64_t to = dst * per_row + in_row;
    *reinterpret_cast<uint2*>((is_v ? a.v[layer] : a.k[layer]) + to * 8) = make_uint2(q.code[0], q.code[1]);
    (is_v ? a.v_group[layer] : a.k_group[layer])[to] = (uint8_t)q.scale;
    if (VALUES) {
        uint16_t* out = is_v ? a.v_round[layer] : a.k_round[layer];
        if (out != nullptr) {
            uint4* p = reinterpret_cast<uint4*>(out + ((int64_t)row * per_row + in_row) * kFp4Group);
            p[0] = make_uint4(q.value[0], q.value[1], q.value[2], q.value[3]);
            p[1] = make_uint4(q.value[4], q.value[5], q.value[6], q.value[7]);
        }
    }
}

}  // namespace

cudaError_t launch_store_fp4(const StoreFp4Args& a, cudaStream_t stream) {
    const int64_t groups = (int64_t)a.n_rows * a.H_kv * kFp4Groups;
    const dim3 grid((unsigned)((groups + kStThreads - 1) / kStThreads), (unsigned)(2 * a.layers));
    return launch_pdl(a.values ? store_fp4_kernel<true> : store_fp4_kernel<false>, grid, dim3(kStThreads), 0, stream,
                      0, a);
}

}  // namespace lsa
