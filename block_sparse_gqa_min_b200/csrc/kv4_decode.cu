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
//    at the running maximum) plus, for fp32 outputs, the f16 of what that rounding left: bf16 outputs
//    round at 2^-9, the f16 of P at 2^-12.
// Every warp works alone: it walks strips of 32 tokens (4608 bytes, one bulk copy each) through a
// ring of its own, so no warp waits for another until the merge.
#include <math.h>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.cuh"

namespace sba {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kRing = kWarps * kStages * kStripBytes;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRowStride = kHeadDim + 4;  // floats between rows of the merge buffer
constexpr float kPShift = 8.f;            // P is exp2(s - max + 8): small weights stay normal f16 numbers
constexpr float kSlack = 7.f;             // the running maximum moves only when exceeded by 2^7 (P <= 2^15)

struct Args {
    const uint8_t* kv;
    const int32_t* block_table;
    const int32_t* seq_lens;
    int32_t* status;
    int H_q, H_kv, b, max_blocks, num_pages, M, rows;  // rows = M * G
    const __nv_bfloat16* q;
    const int32_t* sel_idx;
    const int32_t* sel_cnt;
    int n_max;
    float scale_log2;  // softmax scale * log2(e)
    int splits, row_groups;
    void* out;
    int out_bf16;
    float* lse_out;
    uint32_t* counters;  // [B][H_kv * row_groups]
    float* part_ml;      // [unit][split][R][2]
    float* part_o;       // [unit][split][R][128], unnormalised
};

// Row r of an MMA tile of 16 tokens holds token perm(r): lane i of a quad then finds the four tokens
// of its value operand (rows 2i, 2i+1, 2i+8, 2i+9) next to each other, and neighbouring quads start
// in different halves of the shared-memory banks.
__device__ __forceinline__ int perm(int r) {
    const int i = (r & 7) >> 1;
    return 4 * i + (r >> 3) * 2 + ((r & 1) ^ (i & 1));
}

// One strip from global memory into `dst`, completing on `bar` (16-byte aligned both sides).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

template <int NH>
struct State {
    float o[NH][8][4];  // O^T: [row tile][channel pair mt]: channels 16(lane/4) + 2mt (c0, c1) and + 1 (c2, c3) of
                        // rows 8nh + 2(lane%4) + x
    float m[NH][2], l[NH][2];
    float sc[NH][2];   // softmax scale * log2(e) * 2^e of the row
    int lim[NH][2];    // tokens the row sees
};

template <int NH, bool kSplitP>
__device__ __forceinline__ void attend_strip(State<NH>& st, const uint32_t (&qb)[NH][8][2], uint8_t* strip, int tok0,
                                             int valid, int first_hidden, int lane) {
    const int tr = lane >> 2, i = lane & 3;
    if (valid < kStripTokens) {
        // rows past the last token may hold anything: a scale of 0 makes them 0
        for (int e = lane; e < (kStripTokens - valid) * 8; e += 32)
            strip[kStripKS + valid * 8 + e] = strip[kStripVS + valid * 8 + e] = 0;
        fence_proxy_async_smem();
        __syncwarp();
    }
    if (first_hidden < tok0 + valid) {
        // some rows do not see the last tokens: a NaN among those tokens' values must reach only the
        // rows that do (0 * NaN is NaN in the product below), so it is put there by hand
        const int t0 = max(0, first_hidden - tok0);
        for (int t = t0; t < valid; ++t)
            if (strip[kStripVS + t * 8 + tr] == kScaleNaN) {
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
            if (strip[kStripVS + e] == kScaleNaN) strip[kStripVS + e] = 0;
        fence_proxy_async_smem();
        __syncwarp();
    }
    // ---- S^T = K Q^T: two tiles of 16 tokens ----
    float s[NH][2][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
        const int ra = 16 * mt + perm(tr), rb = 16 * mt + perm(tr + 8);
        const uint4 ka = *reinterpret_cast<const uint4*>(strip + ra * 64 + i * 16);
        const uint4 kb = *reinterpret_cast<const uint4*>(strip + rb * 64 + i * 16);
        const uint32_t sa = *reinterpret_cast<const uint16_t*>(strip + kStripKS + ra * 8 + 2 * i);
        const uint32_t sb = *reinterpret_cast<const uint16_t*>(strip + kStripKS + rb * 8 + 2 * i);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
        const uint32_t fa[2] = {scale_f16x2(sa & 0xff), scale_f16x2(sa >> 8)};
        const uint32_t fb[2] = {scale_f16x2(sb & 0xff), scale_f16x2(sb >> 8)};
        float even[NH][4], odd[NH][4];  // two independent accumulator chains
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int x = 0; x < 4; ++x) even[nh][x] = odd[nh][x] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t a[4], c[4];
            codes_to_f16(wa[w], a[0], a[1], a[2], a[3]);
            codes_to_f16(wb[w], c[0], c[1], c[2], c[3]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                a[x] = mul_f16x2(a[x], fa[w >> 1]);
                c[x] = mul_f16x2(c[x], fb[w >> 1]);
            }
            const uint32_t f0[4] = {a[0], c[0], a[1], c[1]}, f1[4] = {a[2], c[2], a[3], c[3]};
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                mma_f16_16816(even[nh], f0, qb[nh][2 * w][0], qb[nh][2 * w][1]);
                mma_f16_16816(odd[nh], f1, qb[nh][2 * w + 1][0], qb[nh][2 * w + 1][1]);
            }
        }
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int tok = tok0 + (x < 2 ? ra : rb);
                s[nh][mt][x] = tok < st.lim[nh][x & 1] ? (even[nh][x] + odd[nh][x]) * st.sc[nh][x & 1] : -INFINITY;
            }
    }
    // ---- running maximum: moved only when some row's is exceeded by 2^kSlack ----
    float top[NH][2];
    bool grow = false;
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            top[nh][x] = fmaxf(fmaxf(s[nh][0][x], s[nh][0][2 + x]), fmaxf(s[nh][1][x], s[nh][1][2 + x]));
            grow |= top[nh][x] > st.m[nh][x] + kSlack;
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
                    const float alpha = exp2f(st.m[nh][x] - mx);  // 0 from -inf
                    st.m[nh][x] = mx;
                    st.l[nh][x] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                        st.o[nh][mt][x] *= alpha;
                        st.o[nh][mt][2 + x] *= alpha;
                    }
                }
            }
    }
    // ---- P^T as B operands ----
    uint32_t ph[NH][2][2], pl[NH][2][2];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        const float u0 = st.m[nh][0] == -INFINITY ? 0.f : st.m[nh][0] - kPShift;
        const float u1 = st.m[nh][1] == -INFINITY ? 0.f : st.m[nh][1] - kPShift;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            float p[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) p[x] = ex2(s[nh][mt][x] - ((x & 1) ? u1 : u0));
            st.l[nh][0] += p[0] + p[2];
            st.l[nh][1] += p[1] + p[3];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const uint32_t hi = pack_f16(p[2 * hh], p[2 * hh + 1]);
                ph[nh][mt][hh] = movmatrix_trans(hi);
                if (kSplitP) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                    pl[nh][mt][hh] = movmatrix_trans(pack_f16(p[2 * hh] - f.x, p[2 * hh + 1] - f.y));
                }
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
                    if (kSplitP) mma_f16_16816(st.o[nh][4 * w + m], a, pl[nh][mt][0], pl[nh][mt][1]);
                }
            }
        }
    }
}

template <int NH, bool kSplitP>
__global__ void __launch_bounds__(kThreads, NH == 1 ? 2 : 1) decode_kv4_kernel(Args a) {
    constexpr int R = 8 * NH;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ int2 info[kWarps][kStages];  // first token of the strip, valid tokens in it
    __shared__ float ml[kWarps][R][2];
    __shared__ float weight[kWarps][R];
    __shared__ float row_m[R], row_l[R];
    __shared__ int last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sp = blockIdx.x, s = blockIdx.z;
    const int h = blockIdx.y / a.row_groups, rg = blockIdx.y % a.row_groups;
    const int G = a.H_q / a.H_kv;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();

    const int spb = a.b / kStripTokens;  // strips per block
    const int len = max(0, min(__ldca(a.seq_lens + s), a.max_blocks * a.b));
    const int N = blocks_of(len, a.b);
    int nb = N;
    const int32_t* sel = nullptr;
    if (a.sel_idx) {
        nb = __ldca(a.sel_cnt + s * a.H_kv + h);
        if (nb < 0 || nb > a.n_max) {
            if (tid == 0 && sp == 0) report(a.status, SBA_DEV_BAD_SELECTION);
            nb = nb < 0 ? 0 : a.n_max;
        }
        sel = a.sel_idx + ((int64_t)s * a.H_kv + h) * a.n_max;
    }
    const int64_t T = (int64_t)nb * spb;
    const int s0 = (int)(T * sp / a.splits), s1 = (int)(T * (sp + 1) / a.splits);
    const int mine = s0 + warp < s1 ? (s1 - s0 - warp + kWarps - 1) / kWarps : 0;  // strips s0 + warp + kWarps * x
    uint8_t* my_ring = ring + warp * (kStages * kStripBytes);

    // lane x resolves this warp's strip 32 * batch + x
    int64_t src = -1;
    int tok = 0;
    auto resolve = [&](int x) {
        src = -1;
        tok = 0;
        if (x < mine) {
            const int g = s0 + warp + kWarps * x;
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
            const int stage = x % kStages;
            info[warp][stage] = make_int2(t, from >= 0 ? min(kStripTokens, len - t) : 0);
            if (from >= 0) {
                mbar_arrive_expect_tx(&full[warp][stage], kStripBytes);
                bulk_load(my_ring + stage * kStripBytes, a.kv + from, kStripBytes, &full[warp][stage]);
            } else {
                mbar_arrive(&full[warp][stage]);
            }
        }
    };
    for (int x = 0; x < min(mine, kStages); ++x) issue(x);

    // ---- Q: row r of this row group, as f16 scaled to a maximum in [1, 2) ----
    const int tr = lane >> 2, qi = lane & 3;
    State<NH> st;
    uint32_t qb[NH][8][2];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        const int r = rg * R + nh * 8 + tr;
        uint4 w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] = make_uint4(0u, 0u, 0u, 0u);
        if (r < a.rows) {
            const uint4* p = reinterpret_cast<const uint4*>(
                a.q + (((int64_t)s * a.M + r / G) * a.H_q + h * G + r % G) * kHeadDim + 32 * qi);
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = __ldca(p + x);
        }
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
            st.sc[nh][x] = a.scale_log2 * pow2(re);
            st.lim[nh][x] = rr < a.rows ? len - a.M + rr / G + 1 : 0;
            st.m[nh][x] = -INFINITY;
            st.l[nh][x] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) st.o[nh][mt][0] = st.o[nh][mt][1] = st.o[nh][mt][2] = st.o[nh][mt][3] = 0.f;
    }

    const int first_hidden = len - a.M + 1;  // the first token that some row does not see
    for (int x = 0; x < mine; ++x) {
        const int stage = x % kStages;
        if (!mbar_wait(&full[warp][stage], (x / kStages) & 1, a.status)) {
            // give up: nothing of this warp enters the merge, and its copies in flight get the same limit again
            for (int y = x; y < min(mine, x + kStages); ++y) mbar_wait(&full[warp][y % kStages], (y / kStages) & 1, a.status);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                st.m[nh][0] = st.m[nh][1] = -INFINITY;
                st.l[nh][0] = st.l[nh][1] = 0.f;
            }
            break;
        }
        const int2 inf = info[warp][stage];
        if (inf.y > 0)
            attend_strip<NH, kSplitP>(st, qb, my_ring + stage * kStripBytes, inf.x, inf.y, first_hidden, lane);
        __syncwarp();
        if (x + kStages < mine) issue(x + kStages);
    }

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
                ml[warp][r][0] = st.m[nh][x];
                ml[warp][r][1] = l;
            }
        }
    __syncthreads();
    if (tid < R) {
        float m = -INFINITY;
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w][tid][0]);
        float l = 0.f;
        for (int w = 0; w < kWarps; ++w) {
            const float f = ml[w][tid][1] == 0.f ? 0.f : exp2f(ml[w][tid][0] - m);  // a NaN sum stays one
            weight[w][tid] = f;
            l += f * ml[w][tid][1];
        }
        row_m[tid] = m;
        row_l[tid] = l;
    }
    __syncthreads();
    const int64_t unit = ((int64_t)s * a.H_kv + h) * a.row_groups + rg;
    float4 acc[R * 32 / kThreads];
#pragma unroll
    for (int x = 0; x < R * 32 / kThreads; ++x) {
        const int r = (x * kThreads + tid) >> 5, c4 = tid & 31;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < kWarps; ++w) {
            const float f = weight[w][r];
            if (f == 0.f) continue;  // a warp that saw nothing
            const float4 o = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(ring + w * (kStages * kStripBytes)) + r * kRowStride + 4 * c4);
            v.x += f * o.x;
            v.y += f * o.y;
            v.z += f * o.z;
            v.w += f * o.w;
        }
        acc[x] = v;
    }
    if (a.splits > 1) {
        // ---- leave the split's rows; the last CTA of the unit merges them ----
        const int64_t at = (unit * a.splits + sp) * R;
#pragma unroll
        for (int x = 0; x < R * 32 / kThreads; ++x) {
            const int r = (x * kThreads + tid) >> 5, c4 = tid & 31;
            __stcg(reinterpret_cast<float4*>(a.part_o + (at + r) * kHeadDim) + c4, acc[x]);
        }
        if (tid < R) __stcg(reinterpret_cast<float2*>(a.part_ml) + at + tid, make_float2(row_m[tid], row_l[tid]));
        __threadfence();
        __syncthreads();
        if (tid == 0) last = atomicAdd(a.counters + unit, 1u) == (uint32_t)a.splits - 1;
        __syncthreads();
        if (!last) return;
        __threadfence();
        if (tid == 0) a.counters[unit] = 0u;  // ready for the next call
        // weights of the splits, in the ring (splits * R floats fit: checked on the host)
        float* wsp = reinterpret_cast<float*>(ring);
        const float2* mlp = reinterpret_cast<const float2*>(a.part_ml) + unit * a.splits * R;
        for (int r = warp; r < R; r += kWarps) {
            float m = -INFINITY;
            for (int x = lane; x < a.splits; x += 32) m = fmaxf(m, __ldcg(mlp + x * R + r).x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            float l = 0.f;
            for (int x = lane; x < a.splits; x += 32) {
                const float2 p = __ldcg(mlp + x * R + r);
                const float f = p.y == 0.f ? 0.f : exp2f(p.x - m);
                wsp[x * R + r] = f;
                l += f * p.y;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) {
                row_m[r] = m;
                row_l[r] = l;
            }
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < R * 32 / kThreads; ++x) {
            const int r = (x * kThreads + tid) >> 5, c4 = tid & 31;
            const float4* p = reinterpret_cast<const float4*>(a.part_o + (unit * a.splits * R + r) * kHeadDim) + c4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int y = 0; y < a.splits; ++y) {
                const float f = wsp[y * R + r];
                const float4 o = __ldcg(p + (int64_t)y * R * (kHeadDim / 4));
                if (f != 0.f) {
                    v.x += f * o.x;
                    v.y += f * o.y;
                    v.z += f * o.z;
                    v.w += f * o.w;
                }
            }
            acc[x] = v;
        }
    }
#pragma unroll
    for (int x = 0; x < R * 32 / kThreads; ++x) {
        const int r = (x * kThreads + tid) >> 5, c4 = tid & 31, row = rg * R + r;
        if (row >= a.rows) continue;
        const float l = row_l[r];
        const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
        const int64_t orow = ((int64_t)s * a.M + row / G) * a.H_q + h * G + row % G;
        const float4 v = acc[x];
        if (a.out_bf16)
            reinterpret_cast<uint2*>(a.out)[orow * 32 + c4] =
                make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
        else
            reinterpret_cast<float4*>(a.out)[orow * 32 + c4] =
                make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        if (a.lse_out && c4 == 0) a.lse_out[orow] = l == 0.f ? -INFINITY : (row_m[r] - kPShift + log2f(l)) * kLn2;
    }
}

constexpr int kRefSMs = 148;

struct Plan {
    int NH, row_groups, splits;
    size_t counters, ml, total;
};

// Splits: enough CTAs for four waves of two per SM when the sequences are long, so that ragged
// lengths even out, but never fewer than one strip a warp.
Plan plan_of(const sba_cache4& c, int M, int n_max) {
    Plan p;
    const int rows = M * (c.H_q / c.H_kv);
    p.NH = rows <= 8 ? 1 : 2;
    p.row_groups = (rows + 8 * p.NH - 1) / (8 * p.NH);
    const int64_t units = (int64_t)c.B * c.H_kv * p.row_groups;
    const int64_t blocks = n_max > 0 ? n_max : (c.max_len + c.b - 1) / c.b;
    const int64_t strips = blocks * (c.b / kStripTokens);
    int64_t most = (strips + kWarps - 1) / kWarps;
    int64_t want = 2 * kRefSMs / units;
    if (strips >= 64 * kWarps) want = 8 * kRefSMs / units;
    p.splits = (int)(want < 1 ? 1 : want > 128 ? 128 : want);
    if (p.splits > most) p.splits = (int)(most < 1 ? 1 : most);
    const size_t R = 8 * p.NH;
    const size_t rows_all = p.splits > 1 ? (size_t)units * p.splits * R : 0;
    p.counters = 0;
    p.ml = ((size_t)units * 4 + 255) / 256 * 256;
    p.total = p.ml + rows_all * (2 + kHeadDim) * 4;
    return p;
}

template <int NH, bool kSplitP>
int launch_one(const Args& a, dim3 grid, cudaStream_t stream) {
    if (allow_smem<decode_kv4_kernel<NH, kSplitP>>(kRing) != SBA_OK) return SBA_ERR_CUDA;
    return launch(decode_kv4_kernel<NH, kSplitP>, grid, dim3(kThreads), kRing, stream, a);
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
    a.splits = p.splits;
    a.row_groups = p.row_groups;
    a.out = out;
    a.out_bf16 = out_dtype == SBA_OUT_BF16;
    a.lse_out = lse_out;
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.counters = reinterpret_cast<uint32_t*>(w + p.counters);
    a.part_ml = reinterpret_cast<float*>(w + p.ml);
    a.part_o = a.part_ml + (size_t)c.B * c.H_kv * p.row_groups * p.splits * 8 * p.NH * 2;
    dim3 grid(p.splits, c.H_kv * p.row_groups, c.B);
    if (p.NH == 1) return a.out_bf16 ? launch_one<1, false>(a, grid, stream) : launch_one<1, true>(a, grid, stream);
    return a.out_bf16 ? launch_one<2, false>(a, grid, stream) : launch_one<2, true>(a, grid, stream);
}

}  // namespace sba
