// Accumulated attention weights of the cached tokens, per KV head: what an eviction ranks by.
//
//   acc_out[t] = acc_in[t] + sum over rows r of exp((q_r . k_t) * scale + bias_r,j(t) - lse_r)
// over the tokens of the selected blocks (or all blocks), with the rows (token i, head) of the group
// and the log-sum-exp that the attention of the same step returned: the softmax is not formed again,
// so one pass over the keys is enough and every token's sum belongs to one thread (no atomics, the
// same bits on every run).
//
// A warp takes 16 tokens at a time: their keys are the rows of f16/bf16 mma.sync tiles (m16n8k16),
// read straight from global memory into operand registers, with the next tile's keys in flight; the
// query rows are the columns, 8 at a time, kept in shared memory as operand fragments.  The channels
// of an MMA step are permuted alike in both so that every lane's key reads are 16 bytes.
// With few rows the bytes of K bound it: bf16, 8 sequences of 48K, 8 KV heads, 4 rows: 133 us, 93% of the
// copy bandwidth; a gated step's 32 blocks of 64 tokens: 4.5 us.  Many rows, and long four-bit launches, go to
// the second kernel below.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.cuh"
#include "tc.cuh"

namespace sba {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTileTokens = 16;
constexpr int kRowTiles = 8;  // row tiles of 8, all staged at once: 64 rows, 16 KB (more go to the second kernel)
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
    const uint8_t* k;  // bf16 keys or four-bit tiles
    const int32_t* block_table;
    const int32_t* seq_lens;
    int32_t* status;
    int B, H_q, H_kv, b, max_blocks, num_pages, M, rows;
    const __nv_bfloat16* q;
    const int32_t* sel_idx;
    const int32_t* sel_cnt;
    const float* gate_bias;
    int n_max;
    float scale_log2;
    const float* lse;
    const float* acc_in;
    float* acc_out;
};

// The keys of 16 tokens as loaded: lane (tr, i) holds rows tr and tr + 8.
template <bool kFour>
struct Keys;

template <>
struct Keys<false> {  // chunks 4j + i of 8 channels
    uint4 a[4], c[4];
    __device__ __forceinline__ void load(const uint8_t* k, int64_t row, int lane) {
        const uint4* p = reinterpret_cast<const uint4*>(k) + (row + (lane >> 2)) * 16 + (lane & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = ld_once_v4(p + 4 * j);
            c[j] = ld_once_v4(p + 8 * 16 + 4 * j);
        }
    }
    __device__ __forceinline__ void operand(uint32_t (&f)[8][4]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j][0] = a[j].x;
            f[2 * j][1] = c[j].x;
            f[2 * j][2] = a[j].y;
            f[2 * j][3] = c[j].y;
            f[2 * j + 1][0] = a[j].z;
            f[2 * j + 1][1] = c[j].z;
            f[2 * j + 1][2] = a[j].w;
            f[2 * j + 1][3] = c[j].w;
        }
    }
    // first channel of lane quarter i's pair `half` in MMA step ks
    static __device__ __forceinline__ int channel(int ks, int i, int half) {
        return (4 * (ks >> 1) + i) * 8 + 4 * (ks & 1) + 2 * half;
    }
};

template <>
struct Keys<true> {  // channels 32i .. 32i + 31: one 16-byte read a row
    uint4 a, c;
    uint32_t sa, sc;
    __device__ __forceinline__ void load(const uint8_t* k, int64_t row, int lane) {
        // row counts 32 to a strip; a tile of 16 does not leave its strip
        const uint8_t* strip = k + (row >> 5) * kStripBytes;
        const int r = (int)(row & 31) + (lane >> 2), i = lane & 3;
        a = ld_once_v4(strip + r * 64 + i * 16);
        c = ld_once_v4(strip + (r + 8) * 64 + i * 16);
        sa = __ldca(reinterpret_cast<const uint16_t*>(strip + kStripKS + r * 8 + 2 * i));
        sc = __ldca(reinterpret_cast<const uint16_t*>(strip + kStripKS + (r + 8) * 8 + 2 * i));
    }
    __device__ __forceinline__ void operand(uint32_t (&f)[8][4]) const {
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wc[4] = {c.x, c.y, c.z, c.w};
        const uint32_t fa[2] = {scale_f16x2(sa & 0xff), scale_f16x2(sa >> 8)};
        const uint32_t fc[2] = {scale_f16x2(sc & 0xff), scale_f16x2(sc >> 8)};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t x[4], y[4];
            codes_to_f16(wa[w], x[0], x[1], x[2], x[3]);
            codes_to_f16(wc[w], y[0], y[1], y[2], y[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[2 * w + (e >> 1)][2 * (e & 1)] = mul_f16x2(x[e], fa[w >> 1]);
                f[2 * w + (e >> 1)][2 * (e & 1) + 1] = mul_f16x2(y[e], fc[w >> 1]);
            }
        }
    }
    static __device__ __forceinline__ int channel(int ks, int i, int half) { return 32 * i + 4 * ks + 2 * half; }
};

// kShared: a CTA takes an equal share of all units' tiles (a unit being one (sequence, KV head)); else the
// grid is (CTAs a unit, KV heads, sequences).
template <bool kFour, bool kShared>
__global__ void __launch_bounds__(kThreads, 2) accumulate_weights_kernel(Args a) {
    __shared__ uint2 qf[kRowTiles][8][32];
    __shared__ float row_sc[kRowTiles * 8], row_lse[kRowTiles * 8];  // lse in log2 units, or as it is under a bias
    __shared__ int row_lim[kRowTiles * 8];
    __shared__ int tile_plain[kRowTiles];  // every row of the tile is real and has a finite lse

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tr = lane >> 2, qi = lane & 3;
    const int G = a.H_q / a.H_kv;
    pdl_wait();
    pdl_trigger();

    const int tpb = a.b / kTileTokens;
    auto length = [&](int s) { return max(0, min(__ldca(a.seq_lens + s), a.max_blocks * a.b)); };
    auto blocks = [&](int u, int len) {
        if (!a.sel_idx) return blocks_of(len, a.b);
        const int n = __ldca(a.sel_cnt + u);
        if (n < 0 || n > a.n_max) report(a.status, SBA_DEV_BAD_SELECTION);
        return n < 0 ? 0 : min(n, a.n_max);
    };
    int unit = blockIdx.z * gridDim.y + blockIdx.y, at = 0, left = 1;
    if constexpr (kShared) {
        const int ctas = gridDim.x;
        const Share share = share_of(
            a.B * a.H_kv, blockIdx.x, lane, [&](int u) { return blocks(u, a.sel_idx ? 0 : length(u / a.H_kv)) * tpb; },
            [&](int64_t) { return ctas; });
        unit = share.unit;
        at = share.at;
        left = share.left;
    }
    while (left > 0 && unit < a.B * a.H_kv) {
        const int s = kShared ? unit / a.H_kv : (int)blockIdx.z, h = kShared ? unit % a.H_kv : (int)blockIdx.y;
        const int len = length(s), N = blocks_of(len, a.b), nb = blocks(unit, len), T = nb * tpb;
        const int32_t* sel = a.sel_idx ? a.sel_idx + (int64_t)unit * a.n_max : nullptr;
        if constexpr (!kShared) {
            at = (int)((int64_t)T * blockIdx.x / gridDim.x);
            left = (int)((int64_t)T * (blockIdx.x + 1) / gridDim.x) - at;
            if (left == 0) return;
        }
        const int t0 = at, t1 = min(T, at + left);
        const int mine = t0 + warp < t1 ? (t1 - t0 - warp + kWarps - 1) / kWarps : 0;

        // lane x resolves this warp's tile 32 * batch + x: cache row (page, head, row) of its first token
        int64_t row = -1;
        int tok = 0, pos = 0;
        auto resolve = [&](int x) {
            row = -1;
            if (x >= mine) return;
            const int g = t0 + warp + kWarps * x;
            pos = g / tpb;
            const int j = sel ? __ldca(sel + pos) : pos;
            // ascending: a block listed twice would be written by two warps
            if (j < 0 || j >= N || (sel && pos > 0 && __ldca(sel + pos - 1) >= j)) {
                report(a.status, SBA_DEV_BAD_SELECTION);
                return;
            }
            const int64_t page = page_of(a.block_table, a.max_blocks, a.num_pages, s, j, a.status);
            tok = j * a.b + (g % tpb) * kTileTokens;
            if (page >= 0 && tok < len) row = (page * a.H_kv + h) * a.b + (g % tpb) * kTileTokens;
        };

        const int n_tiles = (a.rows + 7) / 8;
        // ---- the rows' operand fragments, scales, lse and limits ----
        if (kShared) __syncthreads();  // the unit before is done with its rows
        for (int t = warp; t < n_tiles; t += kWarps) {
            const int r = t * 8 + tr;
            const bool real = r < a.rows;
            const int64_t qrow = real ? ((int64_t)s * a.M + r / G) * a.H_q + h * G + r % G : 0;
            const __nv_bfloat16* p = a.q + qrow * kHeadDim;
            uint32_t w[8][2];
            float mx = 0.f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t v =
                        real ? __ldca(reinterpret_cast<const uint32_t*>(p + Keys<kFour>::channel(ks, qi, half))) : 0u;
                    w[ks][half] = v;
                    mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(v)), fabsf(bf16_hi(v))));
                }
            float up = 1.f;
            if (kFour) {  // f16 operands: the row scaled by a power of two to a maximum in [1, 2)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const int e = row_exponent(mx);
                const float down = pow2(-e);
                up = pow2(e);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        w[ks][half] = pack_f16(bf16_lo(w[ks][half]) * down, bf16_hi(w[ks][half]) * down);
            }
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) qf[t][ks][lane] = make_uint2(w[ks][0], w[ks][1]);
            const float lse = real ? __ldca(a.lse + qrow) : -INFINITY;
            const bool counts = lse > -INFINITY || lse != lse;  // a row that attended to nothing adds nothing
            if (qi == 0) {
                row_sc[t * 8 + tr] = a.scale_log2 * up;
                row_lse[t * 8 + tr] = !counts ? 0.f : a.gate_bias ? lse : lse * kLog2e;
                row_lim[t * 8 + tr] = counts ? len - a.M + r / G + 1 : 0;
            }
            const int all = __all_sync(0xffffffffu, counts);
            if (lane == 0) tile_plain[t] = all;
        }
        __syncthreads();

        const int first_hidden = len - a.M + 1;
        Keys<kFour> next;
        auto fetch = [&](int x) {
            if ((x & 31) == 0) resolve(x + lane);
            const int64_t from = __shfl_sync(0xffffffffu, row, x & 31);
            if (from >= 0) next.load(a.k, from, lane);
        };
        int64_t cur_row = -1;
        int cur_tok = 0, cur_pos = 0;
        if (mine > 0) fetch(0);
        for (int x = 0; x < mine; ++x) {
            cur_row = __shfl_sync(0xffffffffu, row, x & 31);
            cur_tok = __shfl_sync(0xffffffffu, tok, x & 31);
            cur_pos = __shfl_sync(0xffffffffu, pos, x & 31);
            uint32_t kf[8][4];
            next.operand(kf);
            if (x + 1 < mine) fetch(x + 1);
            if (cur_row < 0) continue;
            float w0 = 0.f, w1 = 0.f;
            const bool all_seen = cur_tok + kTileTokens <= first_hidden;
            for (int t = 0; t < n_tiles; ++t) {
                float e[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < 8; ks += 2) {
                    const uint2 b0 = qf[t][ks][lane], b1 = qf[t][ks + 1][lane];
                    if (kFour) {
                        mma_f16_16816(e, kf[ks], b0.x, b0.y);
                        mma_f16_16816(o, kf[ks + 1], b1.x, b1.y);
                    } else {
                        mma_bf16_16816(e, kf[ks], b0.x, b0.y);
                        mma_bf16_16816(o, kf[ks + 1], b1.x, b1.y);
                    }
                }
                const int r = t * 8 + 2 * qi;
                const float2 sc = *reinterpret_cast<const float2*>(&row_sc[r]);
                float2 off = *reinterpret_cast<const float2*>(&row_lse[r]);
                if (a.gate_bias) {
                    const int64_t at = ((int64_t)s * a.H_q + h * G + r) * a.n_max + cur_pos;
                    // (lse - bias first: where both are the type's lowest value, either in log2 units is infinite)
                    if (r < a.rows) off.x = (off.x - __ldca(a.gate_bias + at)) * kLog2e;
                    if (r + 1 < a.rows) off.y = (off.y - __ldca(a.gate_bias + at + a.n_max)) * kLog2e;
                }
                float p0 = ex2(fmaf(e[0] + o[0], sc.x, -off.x)), p1 = ex2(fmaf(e[1] + o[1], sc.y, -off.y));
                float p2 = ex2(fmaf(e[2] + o[2], sc.x, -off.x)), p3 = ex2(fmaf(e[3] + o[3], sc.y, -off.y));
                if (!all_seen || !tile_plain[t]) {
                    const int2 lim = *reinterpret_cast<const int2*>(&row_lim[r]);
                    if (cur_tok + tr >= lim.x) p0 = 0.f;
                    if (cur_tok + tr >= lim.y) p1 = 0.f;
                    if (cur_tok + tr + 8 >= lim.x) p2 = 0.f;
                    if (cur_tok + tr + 8 >= lim.y) p3 = 0.f;
                }
                w0 += p0 + p1;
                w1 += p2 + p3;
            }
            w0 += __shfl_xor_sync(0xffffffffu, w0, 1);
            w0 += __shfl_xor_sync(0xffffffffu, w0, 2);
            w1 += __shfl_xor_sync(0xffffffffu, w1, 1);
            w1 += __shfl_xor_sync(0xffffffffu, w1, 2);
            if (qi < 2) {  // lane 0 of a quad writes token tr, lane 1 token tr + 8
                const int t = tr + 8 * qi;
                if (cur_tok + t < len) a.acc_out[cur_row + t] = a.acc_in[cur_row + t] + (qi ? w1 : w0);
            }
        }
        if constexpr (!kShared) return;
        left -= t1 - t0;
        at = 0;
        ++unit;
    }
}

// ---------------------------------------------------------------------------
// Many query rows: the products on tcgen05.  A tile of 128 tokens is the MMA's M, 64 query rows its N: a warp
// brings its strip of 32 tokens from codes to f16 and stores it as the A operand in tensor memory, one thread
// issues the eight steps of 16 channels against the rows in shared memory, and every thread reads back the 64
// logits of ONE token, so the sum over the rows is in its own registers (no shuffle, no shared memory).  What
// bounds it is the 16 exponentials a cycle of an SM: 64 rows over 393K tokens and 8 KV heads would take 45 us
// at that rate and take 104 (four bits; 179 in bf16, where the keys alone take 123; 69 in four bits at 4 rows,
// where the bytes would take 38): the unit is 47% busy, since a tile's steps (codes to f16 0.4 us, products
// 0.3, exponentials 0.9) follow one another and tensor memory has room for four tiles an SM.
// Two CTAs of two warpgroups share an SM; every warpgroup works on tiles of its own, so one's conversion
// and its wait for the tensor core overlap the others' exponentials.
// ---------------------------------------------------------------------------
constexpr int kTcThreads = 256;
constexpr int kTcGroups = kTcThreads / 128;
constexpr int kTcChunk = 64;                     // rows of one MMA
constexpr int kTcRows = 256;                     // rows staged at a time
constexpr int kTcSmem = 2 * kTcRows * 128 + 1024;
constexpr uint32_t kTcGroupCols = 128;           // A: 64 columns (f16 pairs), D: 64 (fp32)
constexpr uint32_t kTcCols = kTcGroups * kTcGroupCols;

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

template <bool kFour>
__global__ void __launch_bounds__(kTcThreads, 2) accumulate_weights_tc_kernel(Args a) {
    extern __shared__ uint8_t dyn_raw[];
    uint8_t* qs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
    __shared__ float4 row_p[kTcRows / 2];  // of rows 2r, 2r + 1: their scales, and minus their lse (log2 units)
    __shared__ int row_lim[kTcRows];
    __shared__ int chunk_plain[kTcRows / kTcChunk];  // every real row of the chunk has an lse
    __shared__ uint64_t done[kTcGroups];
    __shared__ uint32_t tmem_at;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.H_q / a.H_kv, spb = a.b / kStripTokens;
    if (tid == 0) {
        for (int i = 0; i < kTcGroups; ++i) mbar_init(&done[i], 1);
        fence_mbar_init();
    }
    if (warp == 0) tc::alloc(&tmem_at, kTcCols);
    pdl_wait();

    // ---- this CTA's share: an equal part of all the units' tiles, whatever their lengths.  A tile is four
    // strips, a unit one (sequence, KV head) ----
    const int units = a.B * a.H_kv;
    auto length = [&](int s) { return max(0, min(__ldca(a.seq_lens + s), a.max_blocks * a.b)); };
    auto blocks = [&](int u) {
        if (!a.sel_idx) return blocks_of(length(u / a.H_kv), a.b);
        const int n = __ldca(a.sel_cnt + u);
        if (n < 0 || n > a.n_max) report(a.status, SBA_DEV_BAD_SELECTION);
        return n < 0 ? 0 : min(n, a.n_max);
    };
    auto tiles = [&](int u) { return (blocks(u) * spb + 3) / 4; };
    const int ctas = gridDim.x;
    const Share share = share_of(units, blockIdx.x, lane, tiles, [&](int64_t) { return ctas; });
    int left = share.left, unit = share.unit, at = share.at;

    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    pdl_trigger();  // not before this CTA holds its tensor memory: the next kernel's CTAs may want some too
    const uint32_t uwarp = tc::uniform(warp), group = uwarp >> 2;
    const uint32_t tm = tc::uniform(tmem_at) + group * kTcGroupCols, my_lanes = (uint32_t)(32 * (uwarp & 3)) << 16;
    const bool issuer = (uwarp & 3) == 0;  // the group's warp that issues its products
    uint32_t phase = 0;
    bool alive = true;

    for (; left > 0 && unit < units; ++unit, at = 0) {
        const int s = unit / a.H_kv, h = unit % a.H_kv;
        const int len = length(s), N = blocks_of(len, a.b), nb = blocks(unit);
        const int32_t* sel = a.sel_idx ? a.sel_idx + (int64_t)unit * a.n_max : nullptr;
        const int t0 = at, n_tiles = min(left, (nb * spb + 3) / 4 - t0);
        left -= n_tiles;
        const int mine = (int)group < n_tiles ? (n_tiles - (int)group + kTcGroups - 1) / kTcGroups : 0;
        const int first_hidden = len - a.M + 1;

        int64_t row = -1;
        int tok = 0;
        auto resolve = [&](int x) {  // lane x: this warp's strip of the group's tile 32 * batch + x
            row = -1;
            tok = 0;
            if (x >= mine) return;
            const int g = 4 * (t0 + (int)group + kTcGroups * x) + (warp & 3), pos = g / spb;
            if (pos >= nb) return;
            const int j = sel ? __ldca(sel + pos) : pos;
            if (j < 0 || j >= N || (sel && pos > 0 && __ldca(sel + pos - 1) >= j)) {
                report(a.status, SBA_DEV_BAD_SELECTION);
                return;
            }
            const int64_t page = page_of(a.block_table, a.max_blocks, a.num_pages, s, j, a.status);
            tok = j * a.b + (g % spb) * kStripTokens;
            if (page >= 0 && tok < len) row = (page * a.H_kv + h) * a.b + (g % spb) * kStripTokens;
        };

        for (int r0 = 0; r0 < a.rows && n_tiles > 0; r0 += kTcRows) {
            const int n_rows = min(kTcRows, a.rows - r0), n_pad = (n_rows + 15) & ~15;
            __syncthreads();  // the rows before are done with
            if (tid < kTcRows / kTcChunk) chunk_plain[tid] = 1;
            __syncthreads();
            Keys<kFour> next[2];
            int64_t from = -1;  // cache row of the strip in hand (four bits: held in `next`), and its first token
            int from_tok = 0;
            auto fetch = [&](int x) {
                if ((x & 31) == 0) resolve(x + lane);
                from = __shfl_sync(0xffffffffu, row, x & 31);
                from_tok = __shfl_sync(0xffffffffu, tok, x & 31);
                if (from < 0) return;
                if (kFour) {
                    next[0].load(a.k, from, lane);
                    next[1].load(a.k, from + 16, lane);
                } else {  // a tile of bf16 keys would take 64 registers: it waits in L2, a row a lane
                    const uint8_t* p = a.k + (from + lane) * (kHeadDim * 2);
                    asm volatile("prefetch.global.L2 [%0];\n\tprefetch.global.L2 [%0+128];" ::"l"(p));
                }
            };
            if (mine > 0) fetch(0);
            // ---- the rows (for four-bit keys as f16, scaled to a maximum in [1, 2) each) in the B operand's
            // layout: 16 lanes a row, lane m the 16-byte chunk m of its 128 positions (64 in each half).
            // Position 16p + 4i + x is channel channel(p, i, 0) + x, the order in which the keys are stored ----
            constexpr int kStep = kTcThreads / 16, kBatch = 4;  // rows of one pass, passes whose loads go together
            const int m = tid & 15, p = m >> 1, i0 = 2 * (m & 1);
            for (int rb = tid >> 4; rb < n_pad; rb += kStep * kBatch) {
                uint2 x0[kBatch], x1[kBatch];
                float lse[kBatch];
#pragma unroll
                for (int y = 0; y < kBatch; ++y) {
                    const int r = rb + y * kStep, gr = r0 + r;
                    x0[y] = x1[y] = make_uint2(0u, 0u);
                    lse[y] = -INFINITY;
                    if (r < n_rows) {
                        const int64_t qrow = ((int64_t)s * a.M + gr / G) * a.H_q + h * G + gr % G;
                        const uint2* src = reinterpret_cast<const uint2*>(a.q + qrow * kHeadDim);
                        x0[y] = __ldca(src + Keys<kFour>::channel(p, i0, 0) / 4);
                        x1[y] = __ldca(src + Keys<kFour>::channel(p, i0 + 1, 0) / 4);
                        lse[y] = __ldca(a.lse + qrow);
                    }
                }
#pragma unroll
                for (int y = 0; y < kBatch; ++y) {
                    const int r = rb + y * kStep;
                    if (r >= n_pad) break;  // the same for a whole warp: n_pad is a multiple of 16
                    const uint32_t w[4] = {x0[y].x, x0[y].y, x1[y].x, x1[y].y};
                    uint32_t f[4] = {w[0], w[1], w[2], w[3]};
                    float up = 1.f;
                    if (kFour) {
                        float mx = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
#pragma unroll
                        for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const int e2 = row_exponent(mx);
                        const float down = pow2(-e2);
                        up = pow2(e2);
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = pack_f16(bf16_lo(w[e]) * down, bf16_hi(w[e]) * down);
                    }
                    *reinterpret_cast<uint4*>(qs + (m >> 3) * (kTcRows * 128) + r * 128 + (((m & 7) ^ (r & 7)) << 4)) =
                        make_uint4(f[0], f[1], f[2], f[3]);
                    if (m == 0) {
                        // a row that attended to nothing adds nothing
                        const bool counts = lse[y] > -INFINITY || lse[y] != lse[y];
                        float* rp = reinterpret_cast<float*>(row_p + r / 2) + (r & 1);
                        rp[0] = counts ? a.scale_log2 * up : 0.f;
                        rp[2] = counts ? -lse[y] * kLog2e : -INFINITY;
                        row_lim[r] = counts ? len - a.M + (r0 + r) / G + 1 : 0;
                        // (a padding row times an infinite bf16 key is a NaN: masked like a row without an lse)
                        if (!counts && (r < n_rows || !kFour)) chunk_plain[r / kTcChunk] = 0;
                    }
                }
            }
            fence_proxy_async_smem();
            __syncthreads();

            const float* acc_from = r0 ? a.acc_out : a.acc_in;
            const uint64_t db = tc::smem_desc(tc::uniform(smem_u32(qs)), 1024);
            for (int x = 0; x < mine; ++x) {
                // ---- the keys to the A operand (a strip that is not there leaves what `next` held: its tokens
                // are not written) ----
                if (!kFour && from >= 0) {
                    next[0].load(a.k, from, lane);
                    next[1].load(a.k, from + 16, lane);
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t f[8][4], v[32];
                    next[half].operand(f);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {  // columns 8ks + 2i, + 1 of rows tr and tr + 8
                        v[4 * ks] = f[ks][0];
                        v[4 * ks + 1] = f[ks][2];
                        v[4 * ks + 2] = f[ks][1];
                        v[4 * ks + 3] = f[ks][3];
                    }
                    tc::st_16x256b_x8(tm + my_lanes + ((uint32_t)(16 * half) << 16), v);
                }
                const int64_t this_row = from + lane;
                const int this_tok = from_tok + lane;
                const bool real = from >= 0 && this_tok < len;
                const float before = real ? acc_from[this_row] : 0.f;
                if (x + 1 < mine) fetch(x + 1);
                tc::wait_st();
                float w = 0.f;
                for (int c0 = 0; c0 < n_rows; c0 += kTcChunk) {
                    const int n = min(kTcChunk, n_pad - c0);
                    // every thread of the group has stored its keys and read its logits of the chunk before
                    tc::fence_before();
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
                    if (issuer && alive) {
                        tc::fence_after();
                        const uint32_t id = tc::idesc(128, n, !kFour), step = (uint32_t)c0 * 128 >> 4;
                        if (tc::elect()) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                tc::mma_ts(tm + 64, tm + 8 * kk,
                                           db + (step + (((kk >> 2) * (kTcRows * 128) + (kk & 3) * 32) >> 4)), id, kk > 0);
                            tc::commit(&done[group]);
                        }
                        __syncwarp();
                    }
                    // a wait that ran out leaves the warp to the barriers only
                    if (alive) alive = mbar_wait_warp(&done[group], phase, a.status);
                    phase ^= 1;
                    tc::fence_after();
                    const bool all_seen = chunk_plain[c0 / kTcChunk] && __all_sync(0xffffffffu, this_tok < first_hidden);
                    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
                    for (int b = 0; b < kTcChunk; b += 32) {
                        if (b >= n) break;
                        // (a chunk of 16 or 48 rows reads 16 columns more than it wrote: what they hold is not used)
                        uint32_t d[32];
                        tc::ld32(tm + 64 + my_lanes + b, d);
                        tc::wait_ld();
                        auto weigh = [&](auto masked, int e0) {
                            const float4* rp = row_p + (c0 + b + e0) / 2;
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float4 q = rp[e >> 1];
                                float2 p = fma2(make_float2(__uint_as_float(d[e0 + e]), __uint_as_float(d[e0 + e + 1])),
                                                make_float2(q.x, q.y), make_float2(q.z, q.w));
                                p.x = ex2(p.x);
                                p.y = ex2(p.y);
                                if (decltype(masked)::value) {
                                    if (this_tok >= row_lim[c0 + b + e0 + e]) p.x = 0.f;
                                    if (this_tok >= row_lim[c0 + b + e0 + e + 1]) p.y = 0.f;
                                }
                                if (e & 2)
                                    sum1 = add2(sum1, p);
                                else
                                    sum0 = add2(sum0, p);
                            }
                        };
                        if (all_seen) {
                            weigh(std::false_type{}, 0);
                            if (b + 16 < n) weigh(std::false_type{}, 16);
                        } else {
                            weigh(std::true_type{}, 0);
                            if (b + 16 < n) weigh(std::true_type{}, 16);
                        }
                    }
                    const float2 sum = add2(sum0, sum1);
                    w += sum.x + sum.y;
                }
                if (real && alive) a.acc_out[this_row] = before + w;
            }
        }
    }
    if (!alive && issuer) mbar_wait_warp(&done[group], phase ^ 1, a.status);  // products still in flight
    tc::fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after();
        tc::dealloc(tmem_at, kTcCols);
    }
}

template <bool kFour, class Cache>
int launch_weights(const Cache& c, const void* keys, const void* q, int M, const int32_t* sel_idx,
                   const int32_t* sel_cnt, const float* gate_bias, int n_max, float scale, const float* lse,
                   const float* acc_in, float* acc_out, cudaStream_t stream) {
    Args a{};
    a.k = static_cast<const uint8_t*>(keys);
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
    a.gate_bias = gate_bias;
    a.n_max = n_max;
    a.scale_log2 = scale * kLog2e;
    a.lse = lse;
    a.acc_in = acc_in;
    a.acc_out = acc_out;
    const int64_t units = (int64_t)c.B * c.H_kv, fit = 2 * 148;
    const int64_t blocks = sel_idx ? n_max : (c.max_len + c.b - 1) / c.b;
    const int64_t tiles = blocks * (c.b / kTileTokens), most = (tiles + kWarps - 1) / kWarps;
    // few tiles (at most four a warp): a CTA works on one unit, which saves the search for its share
    const bool few = units <= fit && units * tiles <= fit * kWarps * 4;
    // Rows from which the tensor-memory kernel is taken, measured on both sides with 8 KV heads (us, mma.sync
    // against tcgen05).  Long launches: four bits, 393K tokens: 4 rows 116 against 71, 64 rows 270 against 104;
    // bf16: 20 rows 162 against 164 (at 24), 32 rows 186 against 161, 64 rows 271 against 183.  A short launch
    // pays for the longer start: four bits, 16K tokens: 16 rows 8.3 against 8.2, 32 rows 10.7 against 9.2; 4K
    // tokens: 32 rows 5.9 against 6.4, 64 rows 8.2 against 7.6; bf16, 16K tokens: 32 rows 11.7 against 13.2,
    // 64 rows 16.2 against 15.2.
    // Gated calls (one token: at most 16 rows) stay with the first kernel, the one that takes a bias.
    static_assert(kMaxGroup <= kRowTiles * 8, "a gated call's rows fit");
    const int least = few ? (kFour ? 24 : kRowTiles * 8) : (kFour ? 1 : 24);
    if (!gate_bias && a.rows >= least) {
        // every CTA that fits (two an SM) once, and at least one tile a warpgroup
        const int64_t wide = (blocks * (c.b / kStripTokens) + 3) / 4, groups = (wide * units + kTcGroups - 1) / kTcGroups;
        if (allow_smem<accumulate_weights_tc_kernel<kFour>>(kTcSmem) != SBA_OK) return SBA_ERR_CUDA;
        return launch(accumulate_weights_tc_kernel<kFour>, dim3((unsigned)(groups < 1 ? 1 : groups < fit ? groups : fit)),
                      dim3(kTcThreads), kTcSmem, stream, a);
    }
    if (few) {
        const int64_t x = fit / units < most ? fit / units : most;
        return launch(accumulate_weights_kernel<kFour, false>, dim3((unsigned)(x < 1 ? 1 : x), c.H_kv, c.B), dim3(kThreads), 0,
                      stream, a);
    }
    // (long four-bit launches have all been taken above, and have no instance here)
    if constexpr (kFour) return SBA_ERR_UNSUPPORTED;
    else return launch(accumulate_weights_kernel<false, true>, dim3((unsigned)fit), dim3(kThreads), 0, stream, a);
}

}  // namespace

int launch_accumulate_weights(const sba_cache& c, const void* q, int M, const int32_t* sel_idx, const int32_t* sel_cnt,
                              const float* gate_bias, int n_max, float scale, const float* lse, const float* acc_in,
                              float* acc_out, cudaStream_t stream) {
    return launch_weights<false>(c, c.k, q, M, sel_idx, sel_cnt, gate_bias, n_max, scale, lse, acc_in, acc_out, stream);
}

int launch_accumulate_weights_kv4(const sba_cache4& c, const void* q, int M, const int32_t* sel_idx,
                                  const int32_t* sel_cnt, int n_max, float scale, const float* lse,
                                  const float* acc_in, float* acc_out, cudaStream_t stream) {
    return launch_weights<true>(c, c.kv, q, M, sel_idx, sel_cnt, nullptr, n_max, scale, lse, acc_in, acc_out, stream);
}

}  // namespace sba
