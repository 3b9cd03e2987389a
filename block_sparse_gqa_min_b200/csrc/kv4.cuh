// The four-bit form of K/V rows, shared by the kernels that write, read and attend to it.
//
// A (page, KV head) tile is b/32 strips of 32 tokens, each 4608 contiguous bytes:
//   key codes [32][64], value codes [32][64], key scales [32][8], value scales [32][8].
// One strip is one bulk copy, and a lane's 16 bytes of a key row are a run of 32 channels.
//
// Codes are e2m1 (sign, two exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), two to a
// byte, the even channel in the low nibble.  A scale byte covers 16 channels and is the top eight
// bits of a positive f16 below its sign (e5m3): scale = f16(byte << 7).  code * scale has at most
// six significant bits and lies in [2^-18, 61440], so it is exact in f16 and in bf16: nothing is
// rounded after the quantisation.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sba {

// Host-side entry points (validated arguments only) of the kernels on four-bit caches and of the
// weights and eviction of either cache.
int check_cache(const sba_cache* c);
int launch_append_kv4(const sba_cache4& c, const void* k_new, const void* v_new, const int32_t* pos_start, int n_new,
                      cudaStream_t stream);
int launch_read_kv4(const sba_cache4& c, const int32_t* pos_start, int n, void* k_out, void* v_out,
                    cudaStream_t stream);
size_t decode_kv4_workspace_bytes(const sba_cache4& c, int M, int n_max);
int launch_decode_kv4(const sba_cache4& c, const void* q, int M, const int32_t* sel_idx, const int32_t* sel_cnt,
                      int n_max, float scale, void* out, int out_dtype, float* lse_out, void* ws,
                      cudaStream_t stream);

int launch_accumulate_weights(const sba_cache& c, const void* q, int M, const int32_t* sel_idx, const int32_t* sel_cnt,
                              const float* gate_bias, int n_max, float scale, const float* lse, const float* acc_in,
                              float* acc_out, cudaStream_t stream);
int launch_accumulate_weights_kv4(const sba_cache4& c, const void* q, int M, const int32_t* sel_idx,
                                  const int32_t* sel_cnt, int n_max, float scale, const float* lse,
                                  const float* acc_in, float* acc_out, cudaStream_t stream);
int launch_evict(const sba_cache& src, const float* acc, const sba_evict_params& p, const sba_cache& dst,
                 float* acc_dst, int32_t* new_lens, int32_t* kept, cudaStream_t stream);
int launch_evict_kv4(const sba_cache4& src, const float* acc, const sba_evict_params& p, const sba_cache4& dst,
                     float* acc_dst, int32_t* new_lens, int32_t* kept, cudaStream_t stream);
int launch_wait_vote_selftest(int32_t* status, int32_t* verdicts, uint64_t limit_ns, cudaStream_t stream);

// mbar_wait by a whole warp, with one verdict: every lane has a clock of its own, and a warp that goes on
// with full-mask operations must not part where the limit runs out for some lanes just before the phase
// completes for the others.  False for all if any lane gave up.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, int32_t* status,
                                               uint64_t limit_ns = kWaitTimeoutNs) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, limit_ns));
}

// 16 bytes that are read once: not kept in L1, and (volatile) never moved above griddepcontrol.wait.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// An equal share of all the units' work for each of `ctas` CTAs, whatever the units' lengths: units are
// laid end to end (unit u has work(u) >= 0 pieces), and CTA c takes pieces [all*c/ctas, all*(c+1)/ctas).
// ctas(all) says among how many CTAs the work is shared, the others get none.  By one whole warp.
struct Share {
    int64_t all;    // pieces of all units
    int64_t start;  // first piece of this share
    int left;       // pieces of it
    int ctas;
    int unit, at;   // the first piece: its unit, and its place in that unit
};
template <class Work, class Ctas>
__device__ __forceinline__ Share share_of(int units, int cta, int lane, Work work, Ctas ctas) {
    Share r;
    const int first = lane < units ? work(lane) : 0;
    int64_t all = first;
    for (int u = 32 + lane; u < units; u += 32) all += work(u);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    r.all = all;
    r.ctas = ctas(all);
    r.start = cta < r.ctas ? all * cta / r.ctas : all;
    r.left = cta < r.ctas ? (int)(all * (cta + 1) / r.ctas - r.start) : 0;
    r.unit = r.at = 0;
    if (r.left == 0) return r;
    int64_t at = r.start;
    for (; r.unit < units; r.unit += 32) {
        const int mine = r.unit == 0 ? first : r.unit + lane < units ? work(r.unit + lane) : 0;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, at < upto);
        if (past) {
            const int x = __ffs(past) - 1;
            r.unit += x;
            r.at = (int)(at - __shfl_sync(0xffffffffu, upto - mine, x));
            return r;
        }
        at -= __shfl_sync(0xffffffffu, upto, 31);
    }
    r.left = 0;  // (the lengths changed while they were being added up)
    return r;
}

// 2^x; results below the normal range become 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// D(16x8 fp32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Power of two that brings a row whose largest magnitude is mx to a maximum in [1, 2), as its
// exponent e (x * 2^-e), within the exponents whose powers and reciprocals are normal numbers: a row of the
// largest bf16 values comes to [2, 4), one of the smallest subnormals to 2^-7 and more.  Rows of zeros,
// infinities and NaN get one that changes nothing else.
__device__ __forceinline__ int row_exponent(float mx) {
    return max(-126, min(126, (int)(__float_as_uint(mx) >> 23) - 127));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Physical page of logical block j of sequence s, or -1 (and a status bit) when the table entry is
// out of range.
__device__ __forceinline__ int64_t page_of(const int32_t* block_table, int max_blocks, int num_pages, int s, int j,
                                           int32_t* status) {
    const int64_t at = (int64_t)s * max_blocks + j;
    const int64_t p = block_table ? (int64_t)__ldca(block_table + at) : at;
    if (p < 0 || p >= num_pages) {
        report(status, SBA_DEV_BAD_PAGE);
        return -1;
    }
    return p;
}

constexpr int kStripTokens = 32;
constexpr int kStripV = 2048;    // value codes
constexpr int kStripKS = 4096;   // key scales
constexpr int kStripVS = 4352;   // value scales
constexpr int kStripBytes = 4608;
constexpr uint32_t kScaleMaxByte = 226;  // 10240: 6 * 10240 still fits f16
constexpr uint32_t kScaleNaN = 0xff;     // a group that held a NaN or an infinity reads back as NaN
constexpr uint32_t kScaleInf = 0xf8;     // from here on bytes are no numbers (infinity, NaN); only kScaleNaN is given out

// Eight codes -> eight f16 (pairs of neighbouring channels, the even one in the low half).
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
        : "r"(w));
}

// A scale byte in both halves of an f16x2.
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t byte) { return byte * 0x00800080u; }

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// f16x2 -> bf16x2, exact for code * scale.
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t a) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a));
    return pack_bf16(f.x, f.y);
}

// Sixteen bf16 channels (x: eight bf16x2) -> eight code bytes and the scale byte.
//
// The scale is the smallest e5m3 value >= amax / 6.  amax has 8 significant bits and 6s at most 6,
// so amax / 6 is either s exactly (and the fp32 quotient is too) or at least 2^-9 away from it
// relatively: rounding the fp32 quotient up gives the exact answer.
// The codes are x / s rounded to the nearest code, ties to the even one.  x * (1/s) in fp32 is
// within 2^-20 of x / s for |x / s| <= 6.  x / s is either one of the tie points .25 .75 1.25 1.75
// 2.5 3.5 5 or at least 2^-10 away from each (x has 8 significant bits, s has 4).  Snapping the
// product to a multiple of 2^-12 therefore lands on a tie point exactly when x / s is one, and
// moves nothing across one.
__device__ __forceinline__ void quantise16(const uint32_t (&x)[8], uint2& codes, uint32_t& scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, x[i] & 0x7fff7fffu);  // |bf16| orders as its bits
    m = max(m & 0xffffu, m >> 16);
    if (m >= 0x7f80u) {  // an infinity or a NaN in the group
        codes = make_uint2(0u, 0u);
        scale = kScaleNaN;
        return;
    }
    const float r = __uint_as_float(m << 16) / 6.f;
    const uint32_t bits = __float_as_uint(r);
    const uint32_t byte = r >= 0x1p-14f ? ((bits + 0xfffffu) >> 20) - (112u << 3) : (uint32_t)ceilf(r * 0x1p17f);
    scale = min(byte, kScaleMaxByte);
    const float s = __half2float(__ushort_as_half((unsigned short)(scale << 7)));
    const float inv = scale ? 1.f / s : 0.f;
    constexpr float kSnap = 0x1.8p11f;  // fp32 steps of 2^-12 around it
    uint32_t out[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = __fadd_rn(__fadd_rn(__fmul_rn(bf16_lo(x[4 * w + i]), inv), kSnap), -kSnap);
            y[2 * i + 1] = __fadd_rn(__fadd_rn(__fmul_rn(bf16_hi(x[4 * w + i]), inv), kSnap), -kSnap);
        }
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(out[w])
            : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    }
    codes = make_uint2(out[0], out[1]);
}

}  // namespace sba
