// Attention of M query tokens over a four-bit cache: selected blocks or all of them, split over the
// sequence and merged in the same launch.
//
// "Rectified Sparse Attention for Efficient Long-Sequence Generation", Summary: exact attention over
// the group's selected blocks, shared by its query heads; its references cite Flash-Decoding (split
// the KV range, merge partial results by log-sum-exp) and PagedAttention (block tables).
//
//   l_rt = (q_r . k_t) * scale,   o_r = sum_t softmax_t(l_rt) v_t,   lse_r = log sum_t exp(l_rt)
// with k_t, v_t the rows as held (code * scale, exact in f16) and row r = (token i, head) seeing
// t <= len - M + i.
//
// A row of the cache is 144 bytes instead of 512, so the arithmetic that brings it back to a matrix
// operand is what has to be kept small:
//  - K.Q^T and V^T.P^T run on f16 mma.sync (m16n8k16, fp32 accumulate) with the tokens (channels) as
//    the 16 rows and up to 8 query rows as the columns, so a group of G <= 8 heads costs one MMA per
//    256 cache values.  Codes become f16 with one conversion per two values and one multiply by the
//    scale; neither rounds.
//  - A lane's share of a key row is 32 neighbouring channels (one 16-byte read); the channels of an
//    MMA step are permuted the same way in Q.  A lane's share of a value row is one scale group; two
//    tokens' codes are interleaved as nibbles (four logic operations for eight results) so that the
//    conversion delivers the token pairs that the A operand wants.
//  - Q enters as f16 after each row is scaled by a power of two to a maximum in [1, 2), P as f16 (2^8
//    at the running maximum) plus the f16 of what that rounding left, whatever the output type: with one
//    f16 alone 6-10% of bf16 outputs came out a step beside the rounding of the exact result.
// Every warp works alone: it walks strips of 32 tokens (4608 bytes, one bulk copy each) through a
// ring of its own, so no warp waits for another until the merge.
//
// Measured on B200: all tokens of 8 sequences of 32-64K, 32/8 heads, bf16 out: 113 us, 4.0 TB/s of the
// cache, 61% of the copy bandwidth (103 with one f16 for P; 121 for fp32 out).  690 instructions a
// strip and warp, most of them turning codes into operands, go out at 2.4 a cycle of an SM (of 4): no
// pipe is full (ALU 48%, tensor 33%, memory 45%), and the four warps a scheduler has, each a chain of
// dependent steps, wait for fixed latencies (24% of their time) and for the ALU (16%).  Short launches
// are bound by their dependent steps: 64 blocks of 64 tokens, 8 KV heads: 9.5 us (lookups 1.5, one
// strip 1.8, the warps' merge 1, partials and their count 1, the last CTA's merge 2).
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.cuh"

namespace sba {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kFlush = 2;  // strips after which fp32 outputs move their sums out of the MMA accumulators
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMostParts = 128;           // CTAs a unit on average, at most: merging more takes longer than they save
constexpr int kRowStride = kHeadDim + 4;  // floats between rows of the merge buffer
constexpr float kPShift = 8.f;            // P is exp2((s - max) * scale + 8): small weights stay normal f16 numbers
constexpr float kSlack = 7.f;             // the running maximum moves only when exceeded by 2^7 (P <= 2^15)

struct Args {
    const uint8_t* kv;
    const int32_t* block_table;
    const int32_t* seq_lens;
    int32_t* status;
    int B, H_q, H_kv, b, max_blocks, num_pages, M, rows;  // rows = M * G
    const __nv_bfloat16* q;
    const int32_t* sel_idx;
    const int32_t* sel_cnt;
    int n_max;
    float scale_log2;  // softmax scale * log2(e)
    int row_groups;
    void* out;
    int out_bf16;
    float* lse_out;
    uint32_t* counters;  // parts that have come, by unit ((sequence, KV head, row group)) or, equal shares, by a unit's first CTA
    float* part_ml;      // [part][R][2]; parts: [unit][CTA of it], or (equal shares) [CTA][its first unit's, its last's]
    float* part_o;       // [part][R][128], unnormalised
};

// Row r of an MMA tile of 16 tokens holds token perm(r): lane i of a quad then finds the four tokens
// of its value operand (rows 2i, 2i+1, 2i+8, 2i+9) next to each other, and neighbouring quads start
// in different halves of the shared-memory banks.
__device__ __forceinline__ int perm(int r) {
    const int i = (r & 7) >> 1;
    return 4 * i + (r >> 3) * 2 + ((r & 1) ^ (i & 1));
}

// CTAs of a unit of T strips that has CTAs of its own: a strip a warp (a second round costs 1 us), but no
// more than 32 (the last CTA merges up to 32 parts in one go; 52 parts of one strip a warp took 13.8 us
// where 26 of two take 11.0).
__host__ __device__ __forceinline__ int64_t parts_of(int64_t T) {
    const int64_t most = (T + kWarps - 1) / kWarps, rounds = (most + 31) / 32;
    return (T + kWarps * rounds - 1) / (kWarps * rounds);
}

// One strip from global memory into `dst`, completing on `bar` (16-byte aligned both sides).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// An MMA drops what does not fit its accumulator instead of rounding it, so a long chain of them drifts.  For
// fp32 outputs a lane therefore adds its accumulators to sums of its own in shared memory every kFlush strips.
// Error and time over all tokens of 8 sequences of 32-64K, by kFlush: never 1.3e-6; 8: 7.4e-7, 116 us; 4:
// 4.7e-7, 118; 2: 3.6e-7, 121; 1: 3.2e-7, 129.  The plain fp32 form is 3.9e-7 off.
template <int NH, bool kF32>
struct Layout {
    static constexpr int kStages = kF32 ? 2 : 3;
    static constexpr int kWarpRing = kStages * kStripBytes;
    static constexpr int kSums = kF32 ? NH * 32 * 32 * 4 : 0;  // per warp: [32 NH values][32 lanes]
    static constexpr int kBytes = kWarps * (kWarpRing + kSums);
};

template <int NH>
struct State {
    float o[NH][8][4];  // O^T: [row tile][channel pair mt]: channels 16(lane/4) + 2mt (c0, c1) and + 1 (c2, c3) of
                        // rows 8nh + 2(lane%4) + x
    float m[NH][2];     // running maximum of the unscaled logits
    float l[NH][2];     // this lane's part of the sums
    float high[NH][2];  // unscaled logit past which the maximum moves
    float sc[NH][2];    // softmax scale * log2(e) * 2^e of the row
    int lim[NH][2];     // tokens the row sees
};

template <int NH, bool kF32>
__device__ __forceinline__ void attend_strip(State<NH>& st, const uint32_t (&qb)[NH][8][2], uint8_t* strip, int tok0,
                                             int valid, bool partial, int first_hidden, float* sums, int lane) {
    const int tr = lane >> 2, i = lane & 3;
    // partial: some row does not see some token of the strip
    if (partial && valid < kStripTokens) {
        // rows past the last token may hold anything: a scale of 0 makes them 0
        for (int e = lane; e < (kStripTokens - valid) * 8; e += 32)
            strip[kStripKS + valid * 8 + e] = strip[kStripVS + valid * 8 + e] = 0;
        fence_proxy_async_smem();
        __syncwarp();
    }
    if (partial && first_hidden < tok0 + valid) {
        // some rows do not see the last tokens: a NaN (or infinity) among those tokens' values must reach only the
        // rows that do (0 * NaN is NaN in the product below), so it is put there by hand
        const int t0 = max(0, first_hidden - tok0);
        for (int t = t0; t < valid; ++t)
            if (strip[kStripVS + t * 8 + tr] >= kScaleInf) {
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (tok0 + t < st.lim[nh][x & 1]) st.o[nh][mt][x] = __int_as_float(0x7fc00000);
            }
        __syncwarp();
        for (int e = t0 * 8 + lane; e < valid * 8; e += 32)
            if (strip[kStripVS + e] >= kScaleInf) strip[kStripVS + e] = 0;
        fence_proxy_async_smem();
        __syncwarp();
    }
    // ---- S^T = K Q^T: two tiles of 16 tokens, a chain of eight MMAs each ----
    float s[NH][2][4];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[nh][mt][x] = 0.f;
    uint4 kc[2][2];
    uint32_t kf[2][2][2];  // scales of channels 32i .. + 15 and + 16 .. of the tile's two rows
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int r = 16 * mt + perm(tr + 8 * y);
            kc[mt][y] = *reinterpret_cast<const uint4*>(strip + r * 64 + i * 16);
            const uint32_t f = *reinterpret_cast<const uint16_t*>(strip + kStripKS + r * 8 + 2 * i);
            kf[mt][y][0] = scale_f16x2(f & 0xff);
            kf[mt][y][1] = scale_f16x2(f >> 8);
        }
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            uint32_t a[4], c[4];
            const uint4 ka = kc[mt][0], kb = kc[mt][1];
            codes_to_f16(w == 0 ? ka.x : w == 1 ? ka.y : w == 2 ? ka.z : ka.w, a[0], a[1], a[2], a[3]);
            codes_to_f16(w == 0 ? kb.x : w == 1 ? kb.y : w == 2 ? kb.z : kb.w, c[0], c[1], c[2], c[3]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                a[x] = mul_f16x2(a[x], kf[mt][0][w >> 1]);
                c[x] = mul_f16x2(c[x], kf[mt][1][w >> 1]);
            }
            const uint32_t f0[4] = {a[0], c[0], a[1], c[1]}, f1[4] = {a[2], c[2], a[3], c[3]};
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                mma_f16_16816(s[nh][mt], f0, qb[nh][2 * w][0], qb[nh][2 * w][1]);
                mma_f16_16816(s[nh][mt], f1, qb[nh][2 * w + 1][0], qb[nh][2 * w + 1][1]);
            }
        }
    // ---- masks (rows past the real ones see all where nothing is masked: they are not written) ----
    if (partial) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int tok = tok0 + 16 * mt + perm(tr + (x < 2 ? 0 : 8));
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
                    if (tok >= st.lim[nh][x & 1]) s[nh][mt][x] = -INFINITY;
            }
    }
    // ---- running maximum (of the unscaled logits: the scale is positive), moved only when some row's is
    // exceeded by 2^kSlack ----
    float top[NH][2];
    bool grow = false;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            top[nh][x] = fmaxf(fmaxf(s[nh][0][x], s[nh][0][2 + x]), fmaxf(s[nh][1][x], s[nh][1][2 + x]));
            grow |= top[nh][x] > st.high[nh][x];
        }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float mx = top[nh][x];
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                if (mx > st.m[nh][x]) {
                    const float alpha = exp2f((st.m[nh][x] - mx) * st.sc[nh][x]);  // 0 from -inf
                    st.m[nh][x] = mx;
                    st.high[nh][x] = __fadd_rd(mx, __fdiv_rd(kSlack, st.sc[nh][x]));
                    st.l[nh][x] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                        st.o[nh][mt][x] *= alpha;
                        st.o[nh][mt][2 + x] *= alpha;
                        if (kF32) {  // (not in use, and not read, where the warp has fewer than kFlush strips)
                            sums[((nh * 8 + mt) * 4 + x) * 32] *= alpha;
                            sums[((nh * 8 + mt) * 4 + 2 + x) * 32] *= alpha;
                        }
                    }
                }
            }
    }
    // ---- P^T as B operands ----
    uint32_t ph[NH][2][2], pl[NH][2][2];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        // (s - m) * scale, not s * scale - m: exactly 0 at the maximum, however large the logits are
        const float u0 = st.m[nh][0] == -INFINITY ? 0.f : st.m[nh][0], u1 = st.m[nh][1] == -INFINITY ? 0.f : st.m[nh][1];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            float p[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) p[x] = ex2(fmaf(s[nh][mt][x] - ((x & 1) ? u1 : u0), st.sc[nh][x & 1], kPShift));
            st.l[nh][0] += p[0] + p[2];
            st.l[nh][1] += p[1] + p[3];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const uint32_t hi = pack_f16(p[2 * hh], p[2 * hh + 1]);
                ph[nh][mt][hh] = movmatrix_trans(hi);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                pl[nh][mt][hh] = movmatrix_trans(pack_f16(p[2 * hh] - f.x, p[2 * hh + 1] - f.y));
            }
        }
    }
    // ---- O^T += V^T P^T ----
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
        // rows 2i, 2i+1, 2i+8, 2i+9 of the tile
        const int e = i & 1;
        const int t0 = 16 * mt + 4 * i + e, t1 = 16 * mt + 4 * i + 1 - e;
        const uint8_t* vc = strip + kStripV + tr * 8;
        const uint8_t* vs = strip + kStripVS + tr;
        const uint2 v0 = *reinterpret_cast<const uint2*>(vc + t0 * 64);
        const uint2 v1 = *reinterpret_cast<const uint2*>(vc + t1 * 64);
        const uint2 v2 = *reinterpret_cast<const uint2*>(vc + (t0 + 2) * 64);
        const uint2 v3 = *reinterpret_cast<const uint2*>(vc + (t1 + 2) * 64);
        const uint32_t f01 = ((uint32_t)vs[t0 * 8] << 7) | ((uint32_t)vs[t1 * 8] << 23);
        const uint32_t f23 = ((uint32_t)vs[(t0 + 2) * 8] << 7) | ((uint32_t)vs[(t1 + 2) * 8] << 23);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint32_t x0 = w ? v0.y : v0.x, x1 = w ? v1.y : v1.x, x2 = w ? v2.y : v2.x, x3 = w ? v3.y : v3.x;
            constexpr uint32_t kLow = 0x0f0f0f0fu;
            // byte m: (channel 2m of token a, channel 2m of token b), and the odd channels
            const uint32_t ea = (x0 & kLow) | ((x1 << 4) & ~kLow), oa = ((x0 >> 4) & kLow) | (x1 & ~kLow);
            const uint32_t eb = (x2 & kLow) | ((x3 << 4) & ~kLow), ob = ((x2 >> 4) & kLow) | (x3 & ~kLow);
            uint32_t a0[4], a1[4], a2[4], a3[4];
            codes_to_f16(ea, a0[0], a0[1], a0[2], a0[3]);
            codes_to_f16(oa, a1[0], a1[1], a1[2], a1[3]);
            codes_to_f16(eb, a2[0], a2[1], a2[2], a2[3]);
            codes_to_f16(ob, a3[0], a3[1], a3[2], a3[3]);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t a[4] = {mul_f16x2(a0[m], f01), mul_f16x2(a1[m], f01), mul_f16x2(a2[m], f23),
                                       mul_f16x2(a3[m], f23)};
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) {
                    mma_f16_16816(st.o[nh][4 * w + m], a, ph[nh][mt][0], ph[nh][mt][1]);
                    mma_f16_16816(st.o[nh][4 * w + m], a, pl[nh][mt][0], pl[nh][mt][1]);
                }
            }
        }
    }
}

// Maximum and sum of a row whose parts' (maximum, sum) the lanes hold, and this lane's part's weight.  A part
// that saw nothing has a sum of 0; a NaN sum stays one.
__device__ __forceinline__ void join(float m, float l, float& weight, float& top, float& sum) {
    top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    weight = l == 0.f ? 0.f : exp2f(m - top);
    sum = weight * l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
}

__device__ __forceinline__ void add_weighted(float4& v, float f, float4 o) {
    v.x = fmaf(f, o.x, v.x);
    v.y = fmaf(f, o.y, v.y);
    v.z = fmaf(f, o.z, v.z);
    v.w = fmaf(f, o.w, v.w);
}

// This lane's accumulators into its sums (or, to end with, its sums into the accumulators).
template <int NH>
__device__ __forceinline__ void move_sums(State<NH>& st, float* sums, bool back) {
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float& s = sums[((nh * 8 + mt) * 4 + x) * 32];
                const float all = s + st.o[nh][mt][x];
                st.o[nh][mt][x] = back ? all : 0.f;
                if (!back) s = all;
            }
}

// kShared: a CTA takes an equal share of all units' strips, which may span several units; else the grid
// is (CTAs a unit, KV heads x row groups, sequences) and a CTA works on one unit.
template <int NH, bool kF32, bool kShared>
__global__ void __launch_bounds__(kThreads, NH == 1 ? 2 : 1) decode_kv4_kernel(Args a) {
    using L = Layout<NH, kF32>;
    constexpr int R = 8 * NH, kStages = L::kStages;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ int2 info[kWarps][kStages];  // first token of the strip; valid tokens in it, negative if some row does not see all 32
    __shared__ float ml[kWarps][R][2];
    __shared__ int last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.H_q / a.H_kv, spb = a.b / kStripTokens;  // strips per block
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share of all units' strips (a unit without any counts one, so that its rows get
    // written); no fewer than a strip a warp, and no more than kMostParts CTAs a unit on average ----
    auto length = [&](int s) { return max(0, min(__ldca(a.seq_lens + s), a.max_blocks * a.b)); };
    auto blocks = [&](int s, int h, int len) {
        if (!a.sel_idx) return blocks_of(len, a.b);
        const int n = __ldca(a.sel_cnt + s * a.H_kv + h);
        if (n < 0 || n > a.n_max) report(a.status, SBA_DEV_BAD_SELECTION);
        return n < 0 ? 0 : min(n, a.n_max);
    };
    Share share{};
    const int units = a.B * a.H_kv * a.row_groups;
    if constexpr (kShared) {
        auto strips = [&](int u) {
            u /= a.row_groups;
            return max(1, blocks(u / a.H_kv, u % a.H_kv, a.sel_idx ? 0 : length(u / a.H_kv)) * spb);
        };
        share = share_of(units, blockIdx.x, lane, strips, [&](int64_t all) {
            const int64_t n = min((all + kWarps - 1) / kWarps, (int64_t)units * kMostParts);
            return (int)min(n, (int64_t)gridDim.x);
        });
    }
    uint8_t* my_ring = ring + warp * L::kWarpRing;
    float* sums = reinterpret_cast<float*>(ring + kWarps * L::kWarpRing + warp * L::kSums) + lane;
    int seq = 0;        // strips this warp has been through (their stages and phases)
    bool alive = true;  // no wait of this warp has run out (the same in all lanes)

    int64_t base = kShared ? share.start - share.at : 0;  // first strip of the unit, among all units'
    int left = kShared ? share.left : 1, at = kShared ? share.at : 0, unit = kShared ? share.unit : 0;
    while (left > 0 && unit < units) {
        int s, h, rg = 0;
        if constexpr (kShared) {
            s = unit / (a.H_kv * a.row_groups);
            h = unit / a.row_groups % a.H_kv;
            rg = unit % a.row_groups;
        } else {
            s = blockIdx.z;
            h = blockIdx.y;
            if (a.row_groups > 1) {
                h = blockIdx.y / a.row_groups;
                rg = blockIdx.y % a.row_groups;
            }
            unit = blockIdx.z * gridDim.y + blockIdx.y;
        }
        const int len = length(s), N = blocks_of(len, a.b), nb = blocks(s, h, len), T = max(1, nb * spb);
        // CTAs that work on the unit, if each works on one only
        const int parts1 = kShared ? 0 : min((int)gridDim.x, (int)parts_of(T));
        if constexpr (!kShared) {
            if ((int)blockIdx.x >= parts1) return;
            at = (int)((int64_t)T * blockIdx.x / parts1);
            left = (int)((int64_t)T * (blockIdx.x + 1) / parts1) - at;
        }
        const int32_t* sel = a.sel_idx ? a.sel_idx + ((int64_t)s * a.H_kv + h) * a.n_max : nullptr;
        const int s0 = at, s1 = min(T, at + left);
        const int mine = s0 + warp < s1 && alive ? (s1 - s0 - warp + kWarps - 1) / kWarps : 0;  // strips s0 + warp + kWarps * x

        // lane x resolves this warp's strip 32 * batch + x
        int64_t src = -1;
        int tok = 0;
        auto resolve = [&](int x) {
            src = -1;
            tok = 0;
            const int g = s0 + warp + kWarps * x;
            if (x < mine && g / spb < nb) {
                const int j = sel ? __ldca(sel + g / spb) : g / spb;
                if (j >= 0 && j < N) {
                    const int64_t page = page_of(a.block_table, a.max_blocks, a.num_pages, s, j, a.status);
                    tok = j * a.b + (g % spb) * kStripTokens;
                    if (page >= 0 && tok < len) src = ((page * a.H_kv + h) * spb + g % spb) * (int64_t)kStripBytes;
                } else {
                    report(a.status, SBA_DEV_BAD_SELECTION);
                }
            }
        };
        auto issue = [&](int x) {  // strip x of this warp into its stage
            if ((x & 31) == 0) resolve(x + lane);
            const int64_t from = __shfl_sync(0xffffffffu, src, x & 31);
            const int t = __shfl_sync(0xffffffffu, tok, x & 31);
            if (lane == 0) {
                const int stage = (seq + x) % kStages;
                const int valid = from >= 0 ? min(kStripTokens, len - t) : 0;
                info[warp][stage] = make_int2(t, t + kStripTokens <= len - a.M + 1 ? valid : -valid);
                if (from >= 0) {
                    mbar_arrive_expect_tx(&full[warp][stage], kStripBytes);
                    bulk_load(my_ring + stage * kStripBytes, a.kv + from, kStripBytes, &full[warp][stage]);
                } else {
                    mbar_arrive(&full[warp][stage]);
                }
            }
        };
        // the query rows' loads go out before the strips are looked up
        const int tr = lane >> 2, qi = lane & 3;
        uint4 qw[NH][4];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            const int r = rg * R + nh * 8 + tr;
#pragma unroll
            for (int x = 0; x < 4; ++x) qw[nh][x] = make_uint4(0u, 0u, 0u, 0u);
            if (r < a.rows) {
                const uint4* p = reinterpret_cast<const uint4*>(
                    a.q + (((int64_t)s * a.M + r / G) * a.H_q + h * G + r % G) * kHeadDim + 32 * qi);
#pragma unroll
                for (int x = 0; x < 4; ++x) qw[nh][x] = __ldca(p + x);
            }
        }
        for (int x = 0; x < min(mine, kStages); ++x) issue(x);

        // ---- Q: row r of this row group, as f16 scaled to a maximum in [1, 2) ----
        State<NH> st;
        uint32_t qb[NH][8][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            const uint4 (&w)[4] = qw[nh];
            float mx = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t ws[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
                for (int y = 0; y < 4; ++y) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(ws[y])), fabsf(bf16_hi(ws[y]))));
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int e = row_exponent(mx);
            const float down = pow2(-e);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t ws[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    qb[nh][2 * x + (y >> 1)][y & 1] = pack_f16(bf16_lo(ws[y]) * down, bf16_hi(ws[y]) * down);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int re = __shfl_sync(0xffffffffu, e, (2 * qi + x) * 4);
                const int rr = rg * R + nh * 8 + 2 * qi + x;
                // (a normal number: 0 would make a NaN of the first maximum, -inf, and of what is masked, and infinity
                // one of the maximum itself; logits so small are all alike, and so large one apart)
                st.sc[nh][x] = fminf(fmaxf(a.scale_log2 * pow2(re), FLT_MIN), FLT_MAX);
                st.lim[nh][x] = rr < a.rows ? len - a.M + rr / G + 1 : 0;
                st.m[nh][x] = st.high[nh][x] = -INFINITY;
                st.l[nh][x] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) st.o[nh][mt][0] = st.o[nh][mt][1] = st.o[nh][mt][2] = st.o[nh][mt][3] = 0.f;
        }

        const int first_hidden = len - a.M + 1;  // the first token that some row does not see
        if (kF32 && mine >= kFlush)
#pragma unroll
            for (int e = 0; e < NH * 32; ++e) sums[e * 32] = 0.f;
        for (int x = 0; x < mine; ++x) {
            const int stage = (seq + x) % kStages;
            if (!mbar_wait_warp(&full[warp][stage], ((seq + x) / kStages) & 1, a.status)) {
                // give up: nothing of this warp enters the merge, and its copies in flight get the same limit again
                for (int y = seq + x; y < seq + min(mine, x + kStages); ++y)
                    mbar_wait_warp(&full[warp][y % kStages], (y / kStages) & 1, a.status);
                alive = false;
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) {
                    st.m[nh][0] = st.m[nh][1] = -INFINITY;
                    st.l[nh][0] = st.l[nh][1] = 0.f;
                }
                break;
            }
            const int2 inf = info[warp][stage];
            if (inf.y != 0)
                attend_strip<NH, kF32>(st, qb, my_ring + stage * kStripBytes, inf.x, abs(inf.y), inf.y < 0, first_hidden, sums, lane);
            if (kF32 && x % kFlush == kFlush - 1) move_sums(st, sums, false);
            __syncwarp();
            if (x + kStages < mine) issue(x + kStages);
        }

        seq += mine;
        if (kF32 && mine >= kFlush) move_sums(st, sums, true);

        // ---- merge the warps: each leaves its rows in its own ring ----
        float* mo = reinterpret_cast<float*>(my_ring);
        __syncwarp();
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float l = st.l[nh][x];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int r = nh * 8 + 2 * qi + x;
#pragma unroll
                for (int mt = 0; mt < 8; ++mt)
                    *reinterpret_cast<float2*>(mo + r * kRowStride + 16 * tr + 2 * mt) =
                        make_float2(st.o[nh][mt][x], st.o[nh][mt][2 + x]);
                if (tr == 0) {
                    ml[warp][r][0] = st.m[nh][x] * st.sc[nh][x];
                    ml[warp][r][1] = l;
                }
            }
        __syncthreads();
        // a warp takes row 8x + warp, a lane four of its channels
        bool write = true;
        float4 acc[NH];
        float row_m[NH], row_l[NH];
#pragma unroll
        for (int x = 0; x < NH; ++x) {
            const int r = 8 * x + warp;
            float f;
            const float l = lane < kWarps ? ml[lane % kWarps][r][1] : 0.f;
            join(lane < kWarps ? ml[lane % kWarps][r][0] : -INFINITY, l, f, row_m[x], row_l[x]);
            const uint32_t saw = __ballot_sync(0xffffffffu, l != 0.f);
            acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float fw = __shfl_sync(0xffffffffu, f, w);
                if (saw >> w & 1)  // (a warp that saw nothing left its ring as it was; a NaN counts whatever its weight)
                    add_weighted(acc[x], fw, *reinterpret_cast<const float4*>(
                        reinterpret_cast<const float*>(ring + w * L::kWarpRing) + r * kRowStride + 4 * lane));
            }
        }
        if (s1 - s0 < T) {
            // ---- a part of the unit: leave its rows; the last CTA of the unit to come merges them ----
            const int64_t slot =
                (kShared ? (int64_t)blockIdx.x * 2 + (share.start >= base ? 0 : 1) : (int64_t)unit * gridDim.x + blockIdx.x) * R;
#pragma unroll
            for (int x = 0; x < NH; ++x) {
                const int64_t at_row = slot + 8 * x + warp;
                __stcg(reinterpret_cast<float4*>(a.part_o + at_row * kHeadDim) + lane, acc[x]);
                if (lane == 0) __stcg(reinterpret_cast<float2*>(a.part_ml) + at_row, make_float2(row_m[x], row_l[x]));
            }
            // the CTAs whose shares meet the unit
            int c0 = 0, parts = parts1;
            if constexpr (kShared) {
                c0 = (int)(((base + 1) * share.ctas + share.all - 1) / share.all) - 1;
                parts = (int)(((base + T) * share.ctas + share.all - 1) / share.all) - c0;
            }
            __threadfence();
            __syncthreads();
            uint32_t* counter = a.counters + (kShared ? c0 : unit);  // (two shared units have different first CTAs)
            if (tid == 0) last = atomicAdd(counter, 1u) == (uint32_t)parts - 1;
            __syncthreads();
            write = last;
            if (write) {
                __threadfence();
                if (tid == 0) *counter = 0u;  // ready for the next call
                // part y's rows; a part is its CTA's first unit's, unless the CTA began before the unit (only the first can)
                constexpr int kStep = kShared ? 2 * R : R;
                int64_t row0 = (int64_t)unit * gridDim.x * R, part0 = row0;
                if constexpr (kShared) {
                    row0 = (int64_t)c0 * 2 * R;
                    part0 = row0 + (share.all * c0 / share.ctas >= base ? 0 : R);
                }
                auto row_of = [&](int y) { return y == 0 ? part0 : row0 + (int64_t)y * kStep; };
                float* weights = reinterpret_cast<float*>(my_ring);  // the parts': at most one a CTA
#pragma unroll 1
                for (int x = 0; x < NH; ++x) {
                    const int r = 8 * x + warp;
                    const float2* mlp = reinterpret_cast<const float2*>(a.part_ml) + r;
                    float m = -INFINITY, l = 0.f;
                    if (parts <= 32) {
                        float2 p = make_float2(-INFINITY, 0.f);
                        if (lane < parts) p = __ldcg(mlp + row_of(lane));
                        float f;
                        join(p.x, p.y, f, m, l);
                        weights[lane] = f;
                    } else {
                        for (int y = lane; y < parts; y += 32) m = fmaxf(m, __ldcg(mlp + row_of(y)).x);
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        for (int y = lane; y < parts; y += 32) {
                            const float2 p = __ldcg(mlp + row_of(y));
                            const float f = p.y == 0.f ? 0.f : exp2f(p.x - m);
                            weights[y] = f;
                            l += f * p.y;
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    }
                    __syncwarp();
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float4* op = reinterpret_cast<const float4*>(a.part_o + r * kHeadDim) + lane;
#pragma unroll 8
                    for (int y = 0; y < parts; ++y)
                        add_weighted(v, weights[y], __ldcg(op + row_of(y) * (kHeadDim / 4)));
                    __syncwarp();
                    // (indexed with constants only, so that they stay in registers)
                    if (x == 0) {
                        acc[0] = v;
                        row_m[0] = m;
                        row_l[0] = l;
                    } else {
                        acc[NH - 1] = v;
                        row_m[NH - 1] = m;
                        row_l[NH - 1] = l;
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < NH; ++x) {
            const int row = rg * R + 8 * x + warp;
            if (row >= a.rows || !write) continue;
            const float l = row_l[x];
            const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
            const int64_t orow = ((int64_t)s * a.M + row / G) * a.H_q + h * G + row % G;
            const float4 v = acc[x];
            if (a.out_bf16)
                reinterpret_cast<uint2*>(a.out)[orow * 32 + lane] =
                    make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
            else
                reinterpret_cast<float4*>(a.out)[orow * 32 + lane] =
                    make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            if (a.lse_out && lane == 0)
                a.lse_out[orow] = l == 0.f ? -INFINITY : (row_m[x] - kPShift + log2f(l)) * kLn2;
        }
        if constexpr (!kShared) return;
        left -= s1 - s0;
        at = 0;
        base += T;
        ++unit;
        // the rings go back to the copies
        fence_proxy_async_smem();
        __syncthreads();
    }
}

constexpr int kRefSMs = 148;
constexpr int kCounters = 512;  // 2 * kRefSMs at most are in use

struct Plan {
    int NH, row_groups, parts, ctas;
    size_t ml, o, total;
};

// Every CTA that fits once (two an SM at 8 rows, one at 16).  Few strips (at most four a warp): a CTA
// works on one unit, which saves the search for its share.  Many: equal shares of all units' strips, so
// that ragged lengths cost nothing.
Plan plan_of(const sba_cache4& c, int M, int n_max) {
    Plan p;
    const int rows = M * (c.H_q / c.H_kv);
    p.NH = rows <= 8 ? 1 : 2;
    p.row_groups = (rows + 8 * p.NH - 1) / (8 * p.NH);
    const int64_t units = (int64_t)c.B * c.H_kv * p.row_groups;
    int64_t strips = (int64_t)(n_max > 0 ? n_max : (c.max_len + c.b - 1) / c.b) * (c.b / kStripTokens);
    if (strips < 1) strips = 1;
    const int64_t fit = p.NH == 1 ? 2 * kRefSMs : kRefSMs, most = parts_of(strips);
    if (units <= fit && units * strips <= fit * kWarps * 4) {
        p.parts = (int)(fit / units < most ? fit / units : most);
        p.ctas = (int)units * p.parts;
    } else {
        p.parts = 0;
        p.ctas = (int)fit;
        if (units * strips < fit * kWarps) p.ctas = (int)((units * strips + kWarps - 1) / kWarps);
    }
    const size_t R = 8 * p.NH;
    p.ml = kCounters * 4;  // at the same place whatever the shape: one workspace serves all
    const size_t parts = (size_t)p.ctas * (p.parts ? 1 : 2);
    p.o = p.ml + parts * R * 2 * 4;
    p.total = p.o + parts * R * kHeadDim * 4;
    return p;
}

template <int NH, bool kF32, bool kShared>
int launch_one(const Args& a, const Plan& p, cudaStream_t stream) {
    if (allow_smem<decode_kv4_kernel<NH, kF32, kShared>>(Layout<NH, kF32>::kBytes) != SBA_OK) return SBA_ERR_CUDA;
    const dim3 grid = kShared ? dim3(p.ctas) : dim3(p.parts, a.H_kv * a.row_groups, a.B);
    return launch(decode_kv4_kernel<NH, kF32, kShared>, grid, dim3(kThreads), Layout<NH, kF32>::kBytes, stream, a);
}

template <int NH>
int launch_rows(const Args& a, const Plan& p, cudaStream_t stream) {
    if (p.parts) return a.out_bf16 ? launch_one<NH, false, false>(a, p, stream) : launch_one<NH, true, false>(a, p, stream);
    return a.out_bf16 ? launch_one<NH, false, true>(a, p, stream) : launch_one<NH, true, true>(a, p, stream);
}

}  // namespace

size_t decode_kv4_workspace_bytes(const sba_cache4& c, int M, int n_max) { return plan_of(c, M, n_max).total; }

int launch_decode_kv4(const sba_cache4& c, const void* q, int M, const int32_t* sel_idx, const int32_t* sel_cnt,
                      int n_max, float scale, void* out, int out_dtype, float* lse_out, void* ws,
                      cudaStream_t stream) {
    const Plan p = plan_of(c, M, n_max);
    Args a{};
    a.kv = static_cast<const uint8_t*>(c.kv);
    a.block_table = c.block_table;
    a.seq_lens = c.seq_lens;
    a.status = c.status;
    a.B = c.B;
    a.H_q = c.H_q;
    a.H_kv = c.H_kv;
    a.b = c.b;
    a.max_blocks = c.max_blocks;
    a.num_pages = c.num_pages;
    a.M = M;
    a.rows = M * (c.H_q / c.H_kv);
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.sel_idx = sel_idx;
    a.sel_cnt = sel_cnt;
    a.n_max = n_max;
    a.scale_log2 = scale * kLog2e;
    a.row_groups = p.row_groups;
    a.out = out;
    a.out_bf16 = out_dtype == SBA_OUT_BF16;
    a.lse_out = lse_out;
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.counters = reinterpret_cast<uint32_t*>(w);
    a.part_ml = reinterpret_cast<float*>(w + p.ml);
    a.part_o = reinterpret_cast<float*>(w + p.o);
    return p.NH == 1 ? launch_rows<1>(a, p, stream) : launch_rows<2>(a, p, stream);
}

}  // namespace sba
