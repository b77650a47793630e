// attend_prompt.cu — causal GQA softmax attention of whole prompts (or of
// their newest tokens over a cache) for packed sequences of different lengths,
// every token up to a row's own attended: the dense pass beside the sparse
// one of attend.cu.
//
// Design (B200): S = Q K^T and O += P V on tcgen05.mma (bf16, fp32
// accumulators in tensor memory), persistent CTAs over work items (row tiles of
// a kv head and, for few rows, a split of the keys).
//  * Rows: one tile of 128 rows is T = 128 / G tokens x the G query heads of
//    one kv head, so that all of them share K and V, a short prompt fills its
//    tiles and the causal border wastes at most one 128-key tile per T tokens.
//    A CTA holds two such tiles (their S and O fill the 512 columns of tensor
//    memory): of consecutive tokens, over the same K/V tiles; or, where there
//    are few rows, of the same tokens, over alternate K/V tiles.
//  * Warps 0..3 and 4..7 are the softmax of the two tiles, one thread per row:
//    scores from tensor memory, running maximum and sum in fp32, P back into
//    the columns S came from as bf16, from where the second product reads it.
//    While one tile's softmax runs, the tensor core works for the other. (Two
//    threads per row, with half the keys each and the maximum exchanged
//    through shared memory, were no faster: 1959 against 1929 us for a prompt
//    of 16384 tokens, 32/4 heads.)
//  * Warp 8 wins the items (the grid has a CTA for each; one that runs takes
//    over those that have not started), looks them up, loads Q and a ring of
//    128-key K and V tiles by TMA; warp 9 issues the MMAs. Every role walks the
//    same items, so an item's loads and first products run under the end of the
//    item before.
//  * The output is rescaled only when a row's maximum has risen by more than
//    2^8 over the one in use, with the next tile, or by more than 2^16, at once
//    (P stays below 2^16, sums are fp32): the softmax threads do it themselves,
//    since S of tile j is complete only after P V of the tile before is (one
//    thread issues both, in order).
//  * Masked keys: the scores are replaced by -infinity, so P is 0, but 0 * V
//    is not 0 where V is an infinity or NaN. In tiles that the mask reaches,
//    V rows behind every row of the CTA (other sequences' rows, rows never
//    written) are zeroed in shared memory, and elements that are not finite
//    within the CTA's own tokens are zeroed and added back at the end, by each
//    row that sees them. Warps 10 and 11 clean the tiles beside the first softmax
//    (by the softmax warps, before it: 157 us for 24 ragged prompts, 150 so).
//  * Partials of split keys are combined by prompt_merge_kernel by log-sum-exp.
//  * What bounds it: the chain of one row tile, softmax (1950 cycles), P V (512),
//    the next S (512) and their hand-overs (350), whose tensor part the other row
//    tile's fills to 62%; with long prompts the board's power as well: 16384
//    tokens, 32/4 heads, 1702 us (1292 TFLOP/s) in the first milliseconds, 1969
//    (1117 TFLOP/s) at the 1.52 GHz that a loop of it holds under the 1000 W cap.
//    Short prompts (24 of up to 1500 tokens: 624 TFLOP/s, tensor pipe 40%) add
//    8000 cycles an item for the first S, the masked tile and the output.
//  * Every wait is bounded; on expiry the kernel flags LSA_DEV_TIMEOUT, waits
//    (bounded) for what it issued, frees its tensor memory and returns.
#include "internal.h"
#include "prompt_parts.cuh"
#include "tcgen05.cuh"

namespace lsa {
namespace {

constexpr int kPrD = 128;
constexpr int kPrRows = 128;                         // rows of a tile
constexpr int kPrKeys = 128;                         // keys of a tile
constexpr int kPrSoftmaxWarps = 8;                    // four per row tile
constexpr int kPrThreads = (kPrSoftmaxWarps + 4) * kWarp;
constexpr int kPrStages = 5;                         // K and V tiles in the ring
constexpr uint32_t kHalf = kPrRows * 128;            // 16 KB: 128 rows of 64 channels
constexpr uint32_t kPrTile = 2 * kHalf;              // 32 KB
constexpr uint32_t kTmemS = 0, kTmemO = 256;         // tensor-memory columns: S0, S1, O0, O1
constexpr uint32_t kIdescS = idesc_bf16(128, 128, false), kIdescO = idesc_bf16(128, 128, true);

// The sequence's rows and tokens, checked.
struct PrSeq {
    int row0, n, base;  // first row, rows, tokens before the first row
    int64_t off;
    bool ok;
};
// A work item: up to two row tiles and a range of key tiles, walked from the
// last to the first: step s is key tile hi - 1 - s. Tile w works on the steps
// first[w], first[w] + stride, ... below n.
struct PrItem {
    PrSeq sq;
    int kvh, split;
    int t[2];       // first token (row of the sequence) of each row tile
    int hi, n;      // key tiles [hi - n, hi)
    int see;        // keys that some row of the item sees
    int masked;     // key tiles from here on hold keys that some row does not see
    int first[2], stride;
    int live;       // 1; 0: nothing to do; -1: behind the CTA's last item
};
constexpr int kPrItems = 3;  // items handed out ahead of their use

struct PrShared {
    uint64_t full[kPrStages], empty[kPrStages];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2];
    uint64_t v_raw[kPrStages];  // a V tile that the mask reaches has landed (its `full` comes once it is clean)
    uint64_t drain;
    uint64_t answer_full;
    alignas(16) uint32_t answer[4];        // the next item as it is won
    uint64_t item_full[kPrItems], item_empty[kPrItems];
    alignas(16) PrItem item[kPrItems];     // the items as warp 8 hands them out
    uint32_t tmem;
    int32_t abort;
    int32_t not_finite;          // some item's own V was not all finite
    int32_t cleaned[kPrStages];  // warps that are done with a V tile under the mask
};
constexpr size_t kPrSharedBytes = (sizeof(PrShared) + 1023) / 1024 * 1024;  // the tiles start on 1024 bytes
constexpr size_t kPrSmem = kPrSharedBytes + (size_t)(2 + kPrStages) * kPrTile;
static_assert(kPrSmem <= 227 * 1024, "shared memory of one CTA");
// registers per thread: the launch's 384 x 168, given to the softmax warps by the others
constexpr int kPrRegsSoftmax = 216, kPrRegsRest = 72;
static_assert(32 * kPrSoftmaxWarps * kPrRegsSoftmax + 128 * kPrRegsRest <= kPrThreads * 168, "register split");

struct PrArgs {
    CUtensorMap q, k, v;
    PromptArgs a;
};

__device__ __forceinline__ bool pr_wait(PrShared& sh, uint64_t& bar, uint32_t parity, int32_t* status) {
    if (mbar_wait_bounded(smem_u32(&bar), parity, kWaitLimitNs)) return true;
    flag(status, LSA_DEV_TIMEOUT);
    atomicExch(&sh.abort, 1);
    return false;
}
__device__ __forceinline__ bool pr_aborted(const PrShared& sh) {
    return *reinterpret_cast<const volatile int32_t*>(&sh.abort) != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The largest of three; NaN if one of them is.
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// P of 32 scores as bf16 pairs, and their sum onto sum[0..1]: 2^(z c - mc),
// kPoly of the 16 pairs on the FMA units, beside the special-function unit, whose
// 16 results a clock and SM are half of what the tensor core's tiles ask for. One
// warp a scheduler alone is fastest with 6 pairs (128 columns 967 cycles, 1519
// without, 1217 with 8); two, in the whole kernel, with 4: 16384 tokens, 32/4
// heads 1933 us with 2, 1916 with 4, 1950 with 6, 2100 with 8. A NaN may come out
// as a number.
// 2^x: x = n + f with n = floor(x) (adding 1.5 * 2^23 rounded down leaves n in
// the low bits), 2^f on [0, 1) by the polynomial of degree 4 with the smallest
// largest relative error (3e-6) among those that are 1 at 0 (fitted by
// reweighted least squares), n added to the exponent. x below -127 counts as
// -127, for which the bits are those of 0. The pairs go through it stage by
// stage, with a few of the others' exponentials between the stages: in
// program order pair by pair the same takes 2021 cycles.
constexpr int kPoly = 4;
__device__ __forceinline__ void exp_split(const float (&z)[32], f32x2 c, f32x2 neg_mc, f32x2 (&sum)[2], uint32_t* p) {
    constexpr int kRest = 16 - kPoly, kStages = 7;
    const f32x2 big = pair(12582912.f, 12582912.f), neg_big = pair(-12582912.f, -12582912.f), minus = pair(-1.f, -1.f);
    f32x2 x[16], t[kPoly], f[kPoly], y[kPoly];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fma2(pair(z[2 * i], z[2 * i + 1]), c, neg_mc);
    auto rest = [&](int stage) {  // the exponentials behind this stage
#pragma unroll
        for (int i = 0; i < kRest; ++i)
            if (i >= kRest * (stage - 1) / kStages && i < kRest * stage / kStages) {
                float p0, p1;
                unpair(x[kPoly + i], p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                sum[i & 1] = add2(sum[i & 1], pair(p0, p1));
                p[kPoly + i] = pack_bf16(p0, p1);
            }
    };
#pragma unroll
    for (int i = 0; i < kPoly; ++i) {
        float x0, x1;
        unpair(x[i], x0, x1);
        x[i] = pair(fmaxf(x0, -127.f), fmaxf(x1, -127.f));
    }
    rest(1);
#pragma unroll
    for (int i = 0; i < kPoly; ++i) t[i] = add2_down(x[i], big);
    rest(2);
#pragma unroll
    for (int i = 0; i < kPoly; ++i) f[i] = add2(t[i], neg_big);
    rest(3);
#pragma unroll
    for (int i = 0; i < kPoly; ++i) f[i] = fma2(f[i], minus, x[i]);
#pragma unroll
    for (int i = 0; i < kPoly; ++i) y[i] = fma2(f[i], pair(0.013426685f, 0.013426685f), pair(0.052242473f, 0.052242473f));
    rest(4);
#pragma unroll
    for (int i = 0; i < kPoly; ++i) y[i] = fma2(y[i], f[i], pair(0.2412802f, 0.2412802f));
    rest(5);
#pragma unroll
    for (int i = 0; i < kPoly; ++i) y[i] = fma2(y[i], f[i], pair(0.69304484f, 0.69304484f));
    rest(6);
#pragma unroll
    for (int i = 0; i < kPoly; ++i) y[i] = fma2(y[i], f[i], pair(1.f, 1.f));
    rest(7);
#pragma unroll
    for (int i = 0; i < kPoly; ++i) {
        float t0, t1, y0, y1;
        unpair(t[i], t0, t1);
        unpair(y[i], y0, y1);
        y0 = __uint_as_float(__float_as_uint(y0) + (__float_as_uint(t0) << 23));
        y1 = __uint_as_float(__float_as_uint(y1) + (__float_as_uint(t1) << 23));
        sum[i & 1] = add2(sum[i & 1], pair(y0, y1));
        p[i] = pack_bf16(y0, y1);
    }
}

// Sequence b owns the tile slots from row_offset[b] / Tc + b on: at least
// ceil(rows / Tc) of them, and every slot number below n_rows / Tc + n_seq
// belongs to one sequence.
__device__ __forceinline__ int slot_seq(const int32_t* row_offset, int n_seq, int tc, int slot) {
    return find_last(n_seq, [&](int b) { return row_offset[b] / tc + b <= slot; });
}

__device__ __forceinline__ PrSeq pr_seq(const PromptArgs& a, int b) {
    PrSeq s;
    s.row0 = a.row_offset[b];
    const int end = a.row_offset[b + 1];
    const int len = a.seq_lens[b];
    s.off = a.kv_offset[b];
    s.n = end - s.row0;
    s.base = len - s.n;
    s.ok = s.row0 >= 0 && end <= a.n_rows && s.n <= len && len <= a.max_len && s.off >= 0 && s.off <= a.total_tokens - len;
    return s;
}

// Item i (every lane of the warp calls it). Sequences' tiles come longest first.
__device__ __forceinline__ PrItem pr_item(const PromptArgs& a, int i) {
    PrItem it;
    if (i == 0 && lane_id() == 0 && rows_outside(a.row_offset, a.n_seq, a.n_rows)) flag(a.dev_status, LSA_DEV_BAD_LENGTH);
    it.split = i % a.n_splits;
    it.kvh = i / a.n_splits % a.H_kv;
    const int slot = i / a.n_splits / a.H_kv;
    const int T = a.tile_tokens, tc = a.dual ? T : 2 * T;
    const int seq = slot_seq(a.row_offset, a.n_seq, tc, slot);
    it.sq = pr_seq(a, seq);
    const int local = slot - (it.sq.row0 / tc + seq);
    const int tiles = (it.sq.n + tc - 1) / tc;
    it.live = it.sq.n > 0 && local >= 0 && local < tiles ? 1 : 0;
    if (it.live && !it.sq.ok) {
        if (local == 0 && lane_id() == 0) flag(a.dev_status, LSA_DEV_BAD_LENGTH);
        it.live = 0;
    }
    if (!it.live) return it;
    it.t[0] = (tiles - 1 - local) * tc;
    it.t[1] = a.dual ? it.t[0] : it.t[0] + T;
    const bool two = a.dual || it.t[1] < it.sq.n;
    it.see = it.sq.base + min(it.t[0] + tc, it.sq.n);
    it.masked = (it.sq.base + it.t[0] + 1) / kPrKeys;
    const int nk = (it.see + kPrKeys - 1) / kPrKeys;
    const int lo = (int)((int64_t)nk * it.split / a.n_splits);
    it.hi = (int)((int64_t)nk * (it.split + 1) / a.n_splits);
    it.n = it.hi - lo;
    it.stride = a.dual ? 2 : 1;
    if (a.dual) {
        it.first[0] = 0;
        it.first[1] = 1;
    } else {
        // the first tile may see fewer key tiles than the second
        const int nk0 = (it.sq.base + min(it.t[0] + T, it.sq.n) + kPrKeys - 1) / kPrKeys;
        it.first[0] = min(max(0, it.hi - nk0), it.n);
        it.first[1] = two ? 0 : it.n;
    }
    return it;
}

// The CTA's items: the grid has one CTA per item, the first has its own index,
// the next ones those of CTAs that had not started. Warp 8 wins them, looks
// them up (2000 cycles of dependent loads and divisions) and hands them to the
// other warps through a ring, ahead of their use.
struct PrItems {
    PrShared& sh;
    int32_t* status;
    int n = 0;  // items taken
    // The next item, which stays in its place until done(); NULL: none left, or
    // a wait gave up. The whole warp calls both.
    __device__ __forceinline__ const PrItem* next() {
        const bool ok = pr_wait(sh, sh.item_full[n % kPrItems], (uint32_t)(n / kPrItems) & 1u, status) && !pr_aborted(sh);
        const PrItem* it = &sh.item[n % kPrItems];
        return __all_sync(0xffffffffu, ok && it->live > 0) ? it : nullptr;
    }
    __device__ __forceinline__ void done() {
        __syncwarp();
        if (lane_id() == 0) mbar_arrive(smem_u32(&sh.item_empty[n % kPrItems]));
        ++n;
    }
};

// 32 bytes.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__global__ void __launch_bounds__(kPrThreads, 1) attend_prompt_kernel(const __grid_constant__ PrArgs args) {
    const PromptArgs& a = args.a;
    extern __shared__ __align__(1024) uint8_t pr_raw[];
    const int tid = threadIdx.x, lane = lane_id(), warp = uniform(warp_id());
    const int G = a.G, T = a.tile_tokens;
    PrShared& sh = *reinterpret_cast<PrShared*>(pr_raw);
    const uint32_t sQ = smem_u32(pr_raw) + (uint32_t)kPrSharedBytes, sKV = sQ + 2 * kPrTile;
    if (tid == 0) {
        for (int i = 0; i < kPrStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
            mbar_init(smem_u32(&sh.v_raw[i]), 1);
            sh.cleaned[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.q_full[i]), 1);
            mbar_init(smem_u32(&sh.q_empty[i]), 1);
            mbar_init(smem_u32(&sh.s_full[i]), 1);
            mbar_init(smem_u32(&sh.p_full[i]), kPrSoftmaxWarps / 2);
            mbar_init(smem_u32(&sh.o_full[i]), 1);
        }
        sh.not_finite = 0;
        for (int i = 0; i < kPrItems; ++i) {
            mbar_init(smem_u32(&sh.item_full[i]), 1);
            mbar_init(smem_u32(&sh.item_empty[i]), kPrSoftmaxWarps + 3);
        }
        mbar_init(smem_u32(&sh.answer_full), 1);
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = 0;
        mbar_fence_init();
    }
    if (warp == kPrSoftmaxWarps + 1) tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)sh.tmem);
    pdl_enter();

    if (warp >= kPrSoftmaxWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrRegsRest));
        if (warp == kPrSoftmaxWarps) {
            // ---- TMA: an item's Q tiles, then K and V of its key tiles --------------------
            int loads = 0;              // K/V tiles asked for so far
            int q_uses[2] = {0, 0};
            int asked = 0, handed = 0;  // items asked for, handed out
            bool ok = true;
            auto hand_out = [&](const PrItem& it) {
                const int at = handed % kPrItems;
                if (handed >= kPrItems)
                    ok = ok && __all_sync(0xffffffffu, pr_wait(sh, sh.item_empty[at], (uint32_t)(handed / kPrItems - 1) & 1u, a.dev_status));
                if (!ok) return;
                if (lane == 0) {
                    sh.item[at] = it;
                    mbar_arrive(smem_u32(&sh.item_full[at]));
                }
                ++handed;
            };
            for (int i = (int)blockIdx.x; ok && i >= 0;) {
                const PrItem it = pr_item(a, i);
                if (it.live) hand_out(it);
                // The item after this one is asked for with this one's last two key tiles: a
                // CTA that asks at an item's start takes items that idle ones could start on
                // (24 chunks of up to 527 rows, 8/4 heads: 94 us, so 68).
                auto ask = [&]() {
                    mbar_arrive_expect_tx(smem_u32(&sh.answer_full), 16);
                    try_cancel(smem_u32(sh.answer), smem_u32(&sh.answer_full));
                    ++asked;
                };
                if (lane == 0 && ok && !(it.live && it.n > 0)) ask();
                if (lane == 0 && it.live) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (!ok || it.first[w] >= it.n) continue;
                        if (q_uses[w] > 0 && !pr_wait(sh, sh.q_empty[w], (q_uses[w] - 1) & 1, a.dev_status)) ok = false;
                        ok = ok && !pr_aborted(sh);
                        if (!ok) continue;
                        ++q_uses[w];
                        mbar_arrive_expect_tx(smem_u32(&sh.q_full[w]), (uint32_t)(T * G) * 256u);
                        for (int h = 0; h < 2; ++h)
                            tma_load_4d(sQ + w * kPrTile + h * kHalf, &args.q, 64 * h, 0, it.kvh, it.sq.row0 + it.t[w],
                                        smem_u32(&sh.q_full[w]));
                    }
                    for (int i = 0; ok && i < 2 * it.n; ++i) {
                        if (i == max(0, 2 * it.n - 4)) ask();
                        const int st = loads % kPrStages;
                        if (loads >= kPrStages && !pr_wait(sh, sh.empty[st], (loads / kPrStages + 1) & 1, a.dev_status))
                            ok = false;
                        if (!ok || pr_aborted(sh)) break;
                        const int j = it.hi - 1 - (i >> 1);
                        const int row = (int)(it.sq.off + (int64_t)j * kPrKeys);
                        const uint32_t bar = (i & 1) && j >= it.masked ? smem_u32(&sh.v_raw[st]) : smem_u32(&sh.full[st]);
                        mbar_arrive_expect_tx(bar, kPrTile);
                        for (int h = 0; h < 2; ++h)
                            tma_load_3d(sKV + st * kPrTile + h * kHalf, (i & 1) ? &args.v : &args.k, 64 * h, it.kvh, row, bar);
                        ++loads;
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)(ok && !pr_aborted(sh)), 0) != 0;
                asked = __shfl_sync(0xffffffffu, asked, 0);
                ok = ok && __all_sync(0xffffffffu, pr_wait(sh, sh.answer_full, (uint32_t)(asked - 1) & 1u, a.dev_status));
                if (ok) i = cancelled_cta(smem_u32(sh.answer));
                fence_proxy_async_smem();
                __syncwarp();
            }
            PrItem end;
            end.live = -1;
            hand_out(end);
            if (lane == 0) {  // every issued copy and answer has landed before the CTA can exit
                if (asked > 0) mbar_wait_bounded(smem_u32(&sh.answer_full), (uint32_t)(asked - 1) & 1u, kWaitLimitNs);
                for (int i = loads > kPrStages ? loads - kPrStages : 0; i < loads; ++i)
                    mbar_wait_bounded(smem_u32(&sh.full[i % kPrStages]), (i / kPrStages) & 1, kWaitLimitNs);
                for (int w = 0; w < 2; ++w)
                    if (q_uses[w] > 0) mbar_wait_bounded(smem_u32(&sh.q_full[w]), (q_uses[w] - 1) & 1, kWaitLimitNs);
            }
        } else if (warp == kPrSoftmaxWarps + 1) {
            // ---- MMA issue --------------------------------------------------------------------
            const uint32_t one = elect_one();
            int loads = 0;           // K/V tiles of the items before
            int uses[2] = {0, 0};    // S tiles issued per row tile
            int q_uses[2] = {0, 0};
            bool ok = true, any = false;
            PrItems items{sh, a.dev_status};
            for (const PrItem* at = items.next(); ok && at != nullptr; at = items.next()) {
                const PrItem& it = *at;
                const int n = uniform(it.n), stride = a.dual ? 2 : 1;
                const int first[2] = {uniform(it.first[0]), uniform(it.first[1])};
                auto wait = [&](uint64_t& bar, int parity) {
                    ok = ok && __all_sync(0xffffffffu, pr_wait(sh, bar, (uint32_t)parity, a.dev_status));
                };
                if (n > 0) any = true;
                for (int s = 0; ok && n > 0 && s < n + stride; ++s) {
                    // step s: P V of the tile's step before, then Q K^T of step s
                    const int p = s - stride;
                    const int gk = loads + 2 * s, gv = loads + 2 * p + 1;  // loads of K of step s, V of step p
                    if (s < n) wait(sh.full[gk % kPrStages], gk / kPrStages & 1);
                    if (p >= 0) wait(sh.full[gv % kPrStages], gv / kPrStages & 1);
                    const uint64_t kd = desc_k_major(sKV + (uint32_t)uniform(gk % kPrStages) * kPrTile);
                    const uint64_t vd = desc_mn_major(sKV + (uint32_t)uniform(p >= 0 ? gv % kPrStages : 0) * kPrTile, kHalf);
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (!ok || (stride == 2 && (s & 1) != w)) continue;
                        if (p >= first[w] && p < n) {
                            wait(sh.p_full[w], (uses[w] - 1) & 1);
                            if (!ok) continue;
                            tmem_fence_after();
                            const uint32_t more = p > first[w];
#pragma unroll
                            for (int x = 0; x < 8; ++x)  // 16 keys: 8 tensor-memory columns of P, 2048 bytes of V
                                mma_bf16_ts(one, tmem + kTmemO + 128 * w, tmem + kTmemS + 128 * w + 8 * x,
                                            vd + (uint64_t)(128 * x), kIdescO, x > 0 ? 1u : more);
                            if (s >= n) mma_commit(one, smem_u32(&sh.o_full[w]));
                        }
                        if (s < n && s >= first[w]) {
                            if (s == first[w]) {
                                wait(sh.q_full[w], q_uses[w] & 1);
                                if (!ok) continue;
                                ++q_uses[w];
                            }
                            tmem_fence_after();
                            const uint64_t qd = desc_k_major(sQ + w * kPrTile);
#pragma unroll
                            for (int x = 0; x < 8; ++x) {  // 16 channels: 32 bytes on, the second half 16 KB on
                                const uint64_t at = (uint64_t)((x & 3) * 2 + (x >> 2) * (kHalf >> 4));
                                mma_bf16_ss(one, tmem + kTmemS + 128 * w, qd + at, kd + at, kIdescS, x > 0);
                            }
                            mma_commit(one, smem_u32(&sh.s_full[w]));
                            if (s + stride >= n) mma_commit(one, smem_u32(&sh.q_empty[w]));
                            ++uses[w];
                        }
                    }
                    if (ok && p >= 0) mma_commit(one, smem_u32(&sh.empty[gv % kPrStages]));
                    if (ok && s < n) mma_commit(one, smem_u32(&sh.empty[gk % kPrStages]));
                    if (__any_sync(0xffffffffu, pr_aborted(sh))) ok = false;
                }
                loads = uniform(loads + 2 * n);
                items.done();
            }
            if (any) {
                mma_commit(one, smem_u32(&sh.drain));
                mbar_wait_bounded(smem_u32(&sh.drain), 0, kWaitLimitNs);
            }
        } else {
            // ---- V under the mask: rows behind `see` become zeros, elements that are
            // not finite in rows that some row of the item does not see are zeroed and noted
            const int half = warp - kPrSoftmaxWarps - 2;  // two warps, every other 16 bytes x 32 each
            int loads = 0;
            uint32_t parity = 0;  // of each stage's v_raw
            bool ok = true;
            PrItems items{sh, a.dev_status};
            for (const PrItem* at = items.next(); ok && at != nullptr; at = items.next()) {
                const int n = at->n, hi = at->hi, masked = at->masked, see = at->see, first_key = at->sq.base + at->t[0] + 1;
                for (int s = 0; ok && s < n && hi - 1 - s >= masked; ++s) {
                    const int j = hi - 1 - s, st = (loads + 2 * s + 1) % kPrStages;
                    ok = __all_sync(0xffffffffu, pr_wait(sh, sh.v_raw[st], parity >> st & 1u, a.dev_status) && !pr_aborted(sh));
                    if (!ok) break;
                    parity ^= 1u << st;
                    const uint32_t v = sKV + (uint32_t)(st * kPrTile);
                    const int r_lo = max(0, first_key - j * kPrKeys), r_end = min(kPrKeys, see - j * kPrKeys);
                    uint32_t found = 0;
                    // 16 bytes of 8 rows' worth at a time: a row of 64 channels is 8 pieces
                    for (int i = 8 * r_lo + 32 * half + lane; i < 8 * r_end; i += 64) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t p = v + h * kHalf + 16 * i;
                            uint4 x = ld_shared_v4(p);
                            uint32_t* e = &x.x;
                            uint32_t any = 0;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t bad = ((e[q] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // an exponent of all ones carries
                                any |= bad;
                                e[q] &= ~(((bad >> 15) & 0x00010001u) * 0xffffu);
                            }
                            found |= any;
                            if (any) st_shared_v4(p, x.x, x.y, x.z, x.w);
                        }
                    }
                    for (int i = 8 * max(r_lo, r_end) + 32 * half + lane; i < 8 * kPrKeys; i += 64) {
                        st_shared_v4(v + 16 * i, 0, 0, 0, 0);
                        st_shared_v4(v + kHalf + 16 * i, 0, 0, 0, 0);
                    }
                    if (found) sh.not_finite = 1;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {  // the second of the two warps passes the tile on
                        __threadfence_block();
                        if (atomicAdd(&sh.cleaned[st], 1) == 1) {
                            sh.cleaned[st] = 0;
                            __threadfence_block();
                            mbar_arrive(smem_u32(&sh.full[st]));
                        }
                    }
                    __syncwarp();
                }
                loads += 2 * n;
                items.done();
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrRegsSoftmax));
        // ---- softmax: one thread per row ------------------------------------------------------
        const int w = warp >> 2;
        const int r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // tensor-memory lanes 32 * (warp & 3) on, in bits 16..
        const uint32_t ts = tmem + lanes + kTmemS + 128u * w, to = tmem + lanes + kTmemO + 128u * w;
        const float c = a.scale_log2;
        const f32x2 c2 = pair(c, c);
        bool ok = true;
        int u = 0, outs = 0;  // S tiles and outputs so far
        PrItems items{sh, a.dev_status};
        for (const PrItem* at = items.next(); ok && at != nullptr; at = items.next()) {
            const PrItem& it = *at;
            const int t_w = w ? it.t[1] : it.t[0];
            const int token = t_w + min(r / G, T - 1);
            const int sees = it.sq.base + min(token, it.sq.n - 1) + 1;  // keys of this row
            const int masked = (it.sq.base + t_w + 1) / kPrKeys;
            float m = -INFINITY, l = 0.f;
            const int first = w ? it.first[1] : it.first[0];
            bool pending = false;  // the maximum in use moves to m_next with the next tile
            float m_next = m;
            auto move_max = [&](float to_m, bool scale_o) {
                const float al = to_m == -INFINITY ? 1.f : ex2((m - to_m) * c);
                m = to_m;
                l *= al;
                if (!scale_o) return;
#pragma unroll 1
                for (int q = 0; q < 8; ++q) {
                    float o[16];
                    tmem_load16(to + 16 * q, o);
                    tmem_load_wait(o);
                    uint32_t x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(o[i] * al);
                    tmem_store16(to + 16 * q, x);
                }
            };
            for (int s = first; s < it.n; s += it.stride, ++u) {
                const int j = it.hi - 1 - s;
                ok = __all_sync(0xffffffffu, pr_wait(sh, sh.s_full[w], u & 1, a.dev_status) && !pr_aborted(sh));
                if (!ok) break;
                tmem_fence_after();
                if (pending) move_max(m_next, true);
                pending = false;
                float z[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_load32(ts + 32 * q, z[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_load_wait(z[q]);
                if (j >= masked) {
                    const int lim = sees - j * kPrKeys;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < 32; ++i) z[q][i] = 32 * q + i < lim ? z[q][i] : -INFINITY;
                }
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mx[q] = max3(z[q][0], z[q][1], z[q][2]);
#pragma unroll
                    for (int i = 3; i < 31; i += 2) mx[q] = max3(mx[q], z[q][i], z[q][i + 1]);
                    mx[q] = max3(mx[q], mx[q], z[q][31]);
                }
                const float top = max3(max3(m, mx[0], mx[1]), mx[2], mx[3]);
                // A score that is NaN makes the row NaN, by its sum. (Rows behind the
                // tile's last hold anything and have no say.)
                if (top != top) l = NAN;
                const float mt = top == top && r < T * G ? top : m;
                const float rise = (mt - m) * c;
                // Behind the first tile the maximum in use stays for this one,
                // unless it has risen far.
                const bool now = s == first || __any_sync(0xffffffffu, rise > 16.f);
                if (__any_sync(0xffffffffu, rise > 8.f)) {
                    pending = !now;
                    m_next = mt;
                    if (now) move_max(mt, s > first);
                }
                const float mc = m == -INFINITY ? 0.f : m * c;
                const f32x2 neg_mc = pair(-mc, -mc);
                f32x2 sum[2] = {0, 0};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t p[16];
                    exp_split(z[q], c2, neg_mc, sum, p);
                    tmem_store16(ts + 16 * q, p);
                }
                float l0, l1;
                unpair(add2(sum[0], sum[1]), l0, l1);
                l += l0 + l1;
                tmem_store_wait();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[w]));
            }
            if (!ok) break;
            // ---- output -------------------------------------------------------------------------
            const bool worked = first < it.n;
            if (worked) {
                ok = __all_sync(0xffffffffu, pr_wait(sh, sh.o_full[w], outs & 1, a.dev_status) && !pr_aborted(sh));
                if (!ok) break;
                ++outs;
                tmem_fence_after();
            }
            const bool mine = r < T * G && token < it.sq.n && (worked || a.n_parts > 1);
            const int64_t row = ((int64_t)it.sq.row0 + token) * a.H_q + it.kvh * G + r % G;
            const int part = a.dual ? 2 * it.split + w : it.split;
            const float inv = 1.f / l;
            float o[4][32];
            if (worked) {
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_load32(to + 32 * q, o[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_load_wait(o[q]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[q][i] = 0.f;
            }
            if (*reinterpret_cast<volatile int32_t*>(&sh.not_finite) != 0 && mine && worked) {
                // V elements of the item's own tokens that are not finite, where this row sees them
                for (int key = it.sq.base + it.t[0] + 1; key < sees; ++key) {
                    const int s = it.hi - 1 - key / kPrKeys;  // the step it belongs to, if it is one of this tile's
                    if (s < first || s >= it.n || (s - first) % it.stride != 0) continue;
                    const uint16_t* vr = a.v + (it.sq.off + key) * a.v_stride + (int64_t)it.kvh * kPrD;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float x = __uint_as_float((uint32_t)vr[32 * q + i] << 16);
                            if (!isfinite(x)) o[q][i] += x;
                        }
                }
            }
            if (mine) {
                uint32_t x[8];
                if (a.n_parts == 1) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            x[i] = pack_bf16(o[q >> 1][16 * (q & 1) + 2 * i] * inv, o[q >> 1][16 * (q & 1) + 2 * i + 1] * inv);
                        store32(a.out + row * kPrD + 16 * q, x);
                    }
                    if (a.lse != nullptr) a.lse[row] = (m * c + log2f(l)) * 0.6931471805599453f;
                } else {
                    const int64_t at = (int64_t)part * a.n_rows * a.H_q + row;
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = __float_as_uint(o[q >> 2][8 * (q & 3) + i]);
                        store32(a.part_o + at * kPrD + 8 * q, x);
                    }
                    reinterpret_cast<float2*>(a.part_ml)[at] = make_float2(l == 0.f ? m * c : fmaxf(m * c, -3e38f), l);
                }
            }
            // (the next item's first P V overwrites O once P is passed on, which this warp does after these loads)
            tmem_fence_before();
            items.done();
        }
    }
    pdl_trigger();
    tmem_fence_before();
    __syncthreads();
    if (warp == kPrSoftmaxWarps + 1) {
        tmem_fence_after();
        tmem_free(tmem, 512);
    }
}

// The parts of a (row, query head) by log-sum-exp, `per` warps each (1, 2, 4
// or 8 of the block's 8).
constexpr int kPmWarps = 8;
__global__ void __launch_bounds__(kPmWarps * kWarp) prompt_merge_kernel(const __grid_constant__ PromptArgs a, int per) {
    pdl_enter();
    __shared__ float s_m[kPmWarps], s_den[kPmWarps];
    __shared__ float4 s_acc[kPmWarps][kWarp];
    const int lane = lane_id(), warp = warp_id(), sub = warp % per;
    const int64_t i = (int64_t)blockIdx.x * (kPmWarps / per) + warp / per;  // row * H_q + head
    bool live = i < (int64_t)a.n_rows * a.H_q;
    const int row = live ? (int)(i / a.H_q) : 0;
    // rows of no sequence, or of one that was refused, stay as they were
    const int seq = find_last(a.n_seq, [&](int b) { return a.row_offset[b] <= row; });
    const PrSeq sq = pr_seq(a, seq);
    live = live && sq.ok && row >= sq.row0 && row < sq.row0 + sq.n;
    const int len = sq.base + sq.n;
    const int parts = !live ? 0 : a.part_keys > 0 ? (len + a.part_keys - 1) / a.part_keys : a.n_parts;
    const int64_t step = (int64_t)a.n_rows * a.H_q;
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float m, float l, float4 v) {
        if (m == -INFINITY) return;  // a part without keys
        const float nm = fmaxf(M, m);
        const float so = exp2f(M - nm), sn = exp2f(m - nm);
        den = den * so + l * sn;
        acc.x = acc.x * so + v.x * sn;
        acc.y = acc.y * so + v.y * sn;
        acc.z = acc.z * so + v.z * sn;
        acc.w = acc.w * so + v.w * sn;
        M = nm;
    };
    for (int s0 = 8 * sub; s0 < parts; s0 += 8 * per) {
        float2 ml[8];
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool in = s0 + u < parts;
            ml[u] = in ? __ldcg(reinterpret_cast<const float2*>(a.part_ml) + (s0 + u) * step + i) : make_float2(-INFINITY, 0.f);
            v[u] = in ? __ldcg(reinterpret_cast<const float4*>(a.part_o + ((s0 + u) * step + i) * kPrD) + lane)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) add(ml[u].x, ml[u].y, v[u]);
    }
    if (per > 1) {
        s_acc[warp][lane] = acc;
        if (lane == 0) {
            s_m[warp] = M;
            s_den[warp] = den;
        }
        __syncthreads();
        if (sub == 0)
            for (int w = 1; w < per; ++w) add(s_m[warp + w], s_den[warp + w], s_acc[warp + w][lane]);
    }
    if (!live || sub != 0) return;
    const float inv = 1.f / den;
    reinterpret_cast<uint2*>(a.out + i * kPrD)[lane] =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (lane == 0 && a.lse != nullptr) a.lse[i] = (M + log2f(den)) * 0.6931471805599453f;
}

}  // namespace

PromptPlan plan_prompt(int n_seq, int n_rows, int max_len, int H_q, int H_kv, int num_sms) {
    PromptPlan p;
    p.G = H_q / H_kv;
    p.tile_tokens = kPrRows / p.G;
    const int key_tiles = (int)(((int64_t)max_len + kPrKeys - 1) / kPrKeys);
    auto workspace = [&]() {
        if (p.n_parts == 1) return;
        const size_t rows = (size_t)p.n_parts * n_rows * H_q;
        p.off_ml = rows * kPrD * 4;
        p.ws_bytes = (p.off_ml + rows * 8 + 255) / 256 * 256;
    };
    // A token or two a sequence (16 (row, query head) columns of a kv head or
    // fewer): attend_prompt_few.cu, the keys in parts of equal size: as many
    // CTAs as run at once (two an SM), but four parts of the longest sequence
    // at least (so that long and short ones even out), 128 at most, and 128
    // keys a part. 16 single tokens over up to 3136 tokens, 32/4 heads: 16 us
    // there, 31 us here; 64 over up to 8000: 89 and 201 us. That is the mean: a
    // sequence of more columns gets further CTAs there, which take turns.
    // Up to eight parts are joined in a cluster where all clusters run at once (16
    // tokens over up to 500: 6.5 us, with the merge kernel 7.9; where they do not,
    // finished CTAs wait in the way of others: 64 tokens over up to 500 22.5 and
    // 16.7 us; 9 over up to 1000, eight parts on 97% of the places, 9.8 and 8.2),
    // and parts of up to 256 keys are taken for that (4 over up to 2000: 7.0
    // against 8.6 us).
    p.few = (int64_t)n_rows * p.G <= 16 * (int64_t)n_seq && n_seq <= 65534;
    if (p.few) {
        const int64_t units = (int64_t)n_seq * H_kv;
        int64_t parts = (2 * (int64_t)num_sms + units - 1) / units;
        auto at_once = [&](int64_t n) { return 4 * units * n <= 7 * (int64_t)num_sms; };  // 7 of 8 places: a cluster lies within one GPC
        if (parts > kFewJoined && max_len <= 256 * kFewJoined && at_once(kFewJoined)) parts = kFewJoined;
        parts = parts < 4 ? 4 : parts > 128 ? 128 : parts;
        p.part_keys = (int)((((int64_t)max_len + parts - 1) / parts + 63) / 64 * 64);
        if (p.part_keys < 128) p.part_keys = 128;
        p.n_parts = (int)(((int64_t)max_len + p.part_keys - 1) / p.part_keys);
        // further runs of columns: all there could be (if one sequence had all rows), or as many as run at once
        p.further = (int)(((int64_t)n_rows * p.G - 1) / few_columns(n_seq, n_rows, p.G));
        const int64_t at_a_time = 2 * num_sms / ((int64_t)p.n_parts * H_kv);
        p.helpers = p.further < at_a_time || p.further == 0 ? p.further : at_a_time > 1 ? (int)at_a_time : 1;
        if (p.helpers > 65535 - n_seq) p.helpers = 65535 - n_seq;  // (the grid's third axis holds them behind the sequences)
        if (p.n_parts > kFewJoined || !at_once(p.n_parts)) workspace();
        return p;
    }
    // Few rows a sequence: one row tile holds them, and a CTA's second tile
    // takes every other key tile instead of more rows.
    p.dual = (int64_t)n_rows <= (int64_t)n_seq * p.tile_tokens && key_tiles >= 2 && (int64_t)n_seq * H_kv < num_sms;
    // (sequences with rows have a slot more than tiles at most)
    const int tc = p.dual ? p.tile_tokens : 2 * p.tile_tokens;
    const int64_t slots = n_rows / tc + n_seq;
    const int64_t items = (((int64_t)n_rows + tc - 1) / tc + (n_seq - 1) / 2) * H_kv;  // about those with rows
    // Key splits: as many as give the shortest of (the longest item, or all items
    // over the SMs and the end of the last ones) + the merge, in us: a step of both
    // tiles takes about 1.7, an item's start and end 5, a row's partials are written
    // and read at 2.5 TB/s. At 32/4 heads, measured for 1, 2 and more splits: 353
    // rows each on 15868 tokens, two sequences 218, 129, 137 us (3); 60 each on
    // 8060, four 115, 67, 36 (6), 34 us (8); 3000-token prompts 77 and 161 us.
    const int64_t keys = max_len - (n_rows / n_seq) / 2 > kPrKeys ? max_len - (n_rows / n_seq) / 2 : kPrKeys;
    const double tiles = (double)key_tiles / (p.dual ? 2 : 1);
    const double steps = (double)((keys + kPrKeys - 1) / kPrKeys) / (p.dual ? 2 : 1);
    double best = 0;
    p.n_splits = 1;
    for (int s = 1; s <= 64 && s <= key_tiles; ++s) {
        const int parts = p.dual ? 2 * s : s;
        const double longest = 1.7 * (tiles / s + 0.5) + 5, mean = 1.7 * (steps / s + 0.5) + 5;
        double t = longest;
        if (items * s > num_sms) {
            // the last round is full or empty where items are alike, else short items even it out
            const int64_t rounds = (items * s + num_sms - 1) / num_sms;
            const double all = mean > 0.9 * longest ? (double)rounds * mean : ((double)(items * s) / num_sms + 0.3) * mean;
            if (all > t) t = all;
        }
        if (parts > 1) t += 3 + 2.0 * parts * n_rows * H_q * 520 / 2.5e6;
        if (s == 1 || t < 0.97 * best) {
            best = t;
            p.n_splits = s;
        }
    }
    p.n_parts = p.dual ? 2 * p.n_splits : p.n_splits;
    p.n_items = slots * H_kv * p.n_splits;
    workspace();
    return p;
}

cudaError_t launch_attend_prompt(const PromptArgs& a, const PromptPlan& p, cudaStream_t stream) {
    cudaError_t e;
    if (p.few) {
        e = launch_attend_prompt_few(a, p.n_parts, stream);
    } else {
        PrArgs args;
        args.a = a;
        if (!tensor_map_rows_bf16(&args.q, a.q, a.n_rows, a.H_kv, a.G, a.q_stride, a.tile_tokens) ||
            !tensor_map_rows_bf16(&args.k, a.k, a.total_tokens, a.H_kv, 0, a.k_stride, kPrKeys) ||
            !tensor_map_rows_bf16(&args.v, a.v, a.total_tokens, a.H_kv, 0, a.v_stride, kPrKeys))
            return cudaErrorInvalidValue;
        static std::atomic<uint64_t> allowed{0};
        e = allow_smem(attend_prompt_kernel, kPrSmem, allowed);
        if (e != cudaSuccess) return e;
        e = launch_pdl(attend_prompt_kernel, dim3((unsigned)p.n_items), dim3(kPrThreads), kPrSmem, stream, 0, args);
    }
    if (e != cudaSuccess || p.ws_bytes == 0) return e;
    const int per = p.n_parts <= 8 ? 1 : p.n_parts <= 16 ? 2 : p.n_parts <= 32 ? 4 : 8;  // eight parts in flight a warp
    const int64_t blocks = ((int64_t)a.n_rows * a.H_q + kPmWarps / per - 1) / (kPmWarps / per);
    return launch_pdl(prompt_merge_kernel, dim3((unsigned)blocks), dim3(kPmWarps * kWarp), 0, stream, 0, a, per);
}

}  // namespace lsa
