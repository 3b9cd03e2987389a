// Writing K/V rows into four-bit pages, and reading them back.
//
// "Rectified Sparse Attention for Efficient Long-Sequence Generation", Summary: KV entries and
// block keys are written as decoding goes on and overwritten when a window is re-encoded; here the
// entries are held in four bits (kv4.cuh), and the Quest descriptors are those of the keys as they
// are held, so a block's score bounds the logits that its attention computes.
#include <math.h>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.cuh"

namespace sba {

namespace {

constexpr int kThreads = 256;

// 32 bytes that nothing here reads again, by one load (volatile: never moved above griddepcontrol.wait).
__device__ __forceinline__ void load_once_32(const void* p, uint32_t (&v)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}

// One CTA per (touched block, KV head, sequence).  Thread t owns channels 16(t%8) .. +15 of rows
// t/8, t/8 + 32, ...: one scale group, so a row's codes are 8 lanes x 8 bytes and a thread needs no
// other thread's data but for the descriptors.  The block's other valid rows are read back as held,
// so that an overwrite can lower a max or raise a min.  No other CTA touches this tile.
// 32K tokens x 8 heads: 36 us (172 MB in and out: 4.7 TB/s, 72% of the copy bandwidth; 3.0 instructions a cycle
// of an SM go out, of 4, and the ALU is 59% busy with the codes' arithmetic); one token of 8 sequences: 3 us.
template <int kBlk>
__global__ void __launch_bounds__(kThreads) append_kv4_kernel(sba_cache4 c, const uint4* k_new,
                                                              const uint4* v_new,
                                                              const int32_t* pos_start, int n_new) {
    constexpr int kRows = kBlk / 32;  // rows per thread
    __shared__ __half2 red[kThreads / 32][2][8][8];
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
    const int g = tid & 7, r0 = tid >> 3;
    const int p0 = __ldca(pos_start + s);
    if (p0 < 0 || (int64_t)p0 + n_new > (int64_t)c.max_blocks * kBlk) {
        if (tid == 0 && blockIdx.x == 0 && h == 0) report(c.status, SBA_DEV_BAD_POSITION);
        return;
    }
    const int j = p0 / kBlk + blockIdx.x;
    if (j > (p0 + n_new - 1) / kBlk) return;
    const int len = __ldca(c.seq_lens + s);
    const int64_t page = page_of(c.block_table, c.max_blocks, c.num_pages, s, j, tid == 0 ? c.status : nullptr);
    if (page < 0) return;
    uint8_t* tile = static_cast<uint8_t*>(c.kv) + (page * c.H_kv + h) * (int64_t)(kRows * kStripBytes);

    // every new row's loads, then the old rows' that count in the descriptor, before anything waits for them
    uint32_t x[2][kRows][8];
    uint2 old[kRows];
    uint32_t old_scale[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int t = j * kBlk + i * 32 + r0;
        old[i] = make_uint2(0u, 0u);
        old_scale[i] = 0;
        if (t >= p0 && t < p0 + n_new) {
            const int64_t src = (((int64_t)s * n_new + (t - p0)) * c.H_kv + h) * 16 + 2 * g;
            load_once_32(k_new + src, x[0][i]);
            load_once_32(v_new + src, x[1][i]);
        } else if (c.desc != nullptr && t < len) {
            const uint8_t* strip = tile + i * kStripBytes;
            old[i] = *reinterpret_cast<const uint2*>(strip + r0 * 64 + g * 8);
            old_scale[i] = strip[kStripKS + r0 * 8 + g];
        }
    }
    __half2 mn[8], mx[8];
    const __half2 top = __half2half2(__ushort_as_half(0x7c00)), bottom = __half2half2(__ushort_as_half(0xfc00));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mn[i] = top;
        mx[i] = bottom;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        uint8_t* strip = tile + i * kStripBytes;
        const int t = j * kBlk + i * 32 + r0;
        const bool is_new = t >= p0 && t < p0 + n_new;
        uint2 kc = old[i];
        uint32_t ks = old_scale[i];
        if (is_new) {
            uint2 vc;
            uint32_t vs;
            quantise16(x[0][i], kc, ks);
            quantise16(x[1][i], vc, vs);
            *reinterpret_cast<uint2*>(strip + r0 * 64 + g * 8) = kc;
            *reinterpret_cast<uint2*>(strip + kStripV + r0 * 64 + g * 8) = vc;
            strip[kStripKS + r0 * 8 + g] = (uint8_t)ks;
            strip[kStripVS + r0 * 8 + g] = (uint8_t)vs;
        }
        if (c.desc != nullptr && t < len) {
            uint32_t v[8];
            codes_to_f16(kc.x, v[0], v[1], v[2], v[3]);
            codes_to_f16(kc.y, v[4], v[5], v[6], v[7]);
            const uint32_t sc = scale_f16x2(ks);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t y = mul_f16x2(v[e], sc);
                mn[e] = __hmin2(mn[e], *reinterpret_cast<const __half2*>(&y));
                mx[e] = __hmax2(mx[e], *reinterpret_cast<const __half2*>(&y));
            }
        }
    }
    if (c.desc == nullptr || j * kBlk >= len) return;  // the same for the whole CTA
    // rows of one warp (lanes 8 apart hold the same channels), then the warps
    const int warp = tid >> 5, lane = tid & 31;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            mn[e] = __hmin2(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], o));
            mx[e] = __hmax2(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
        }
        if (lane < 8) {
            red[warp][0][lane][e] = mn[e];
            red[warp][1][lane][e] = mx[e];
        }
    }
    __syncthreads();
    if (tid < 128) {  // thread = (min or max, channel pair)
        const int which = tid >> 6, pair = tid & 63;
        __half2 v = red[0][which][pair >> 3][pair & 7];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) {
            const __half2 x = red[w][which][pair >> 3][pair & 7];
            v = which ? __hmax2(v, x) : __hmin2(v, x);
        }
        reinterpret_cast<uint32_t*>(c.desc)[((page * c.H_kv + h) * 2 + which) * 64 + pair] =
            f16x2_to_bf16x2(*reinterpret_cast<const uint32_t*>(&v));
    }
}

// 32 bytes that nothing here reads again: one store, first to leave L2.
__device__ __forceinline__ void store_once_32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// One CTA per (block that overlaps the window, KV head, sequence).  Thread t owns one scale group (channels
// 16(t%8) .. +15) of rows t/8, t/8 + 32, ...: 8 code bytes and a scale byte in, one 32-byte store out, so a
// row's 256 bytes are written by 8 neighbouring lanes.  Every load of the thread is issued before its first
// store.  262144 tokens x 4 heads: 115 us, 6.0 TB/s in and out, 91% of the copy bandwidth (16 bytes a store
// and the loads of one tensor at a time: 138 us).
template <int kBlk>
__global__ void __launch_bounds__(kThreads) read_kv4_kernel(sba_cache4 c, const int32_t* pos_start, int n,
                                                            uint4* k_out, uint4* v_out) {
    constexpr int kRows = kBlk / 32;
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
    const int g = tid & 7, r0 = tid >> 3;
    const int p0 = __ldca(pos_start + s);
    if (p0 < 0 || (int64_t)p0 + n > (int64_t)c.max_blocks * kBlk) {
        if (tid == 0 && blockIdx.x == 0 && h == 0) report(c.status, SBA_DEV_BAD_POSITION);
        return;
    }
    const int j = p0 / kBlk + blockIdx.x;
    const int end = min(p0 + n, __ldca(c.seq_lens + s));
    if (j * kBlk >= end) return;
    const int64_t page = page_of(c.block_table, c.max_blocks, c.num_pages, s, j, tid == 0 ? c.status : nullptr);
    if (page < 0) return;
    const uint8_t* tile = static_cast<const uint8_t*>(c.kv) + (page * c.H_kv + h) * (int64_t)(kRows * kStripBytes);
    uint2 code[2][kRows];
    uint32_t sc[2][kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int t = j * kBlk + 32 * i + r0;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            code[which][i] = make_uint2(0u, 0u);
            sc[which][i] = 0;
            if (t >= p0 && t < end) {
                const uint8_t* strip = tile + i * kStripBytes;
                code[which][i] = __ldcs(reinterpret_cast<const uint2*>(strip + which * kStripV + r0 * 64 + g * 8));
                sc[which][i] = __ldca(strip + (which ? kStripVS : kStripKS) + r0 * 8 + g);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int t = j * kBlk + 32 * i + r0;
        if (t < p0 || t >= end) continue;
        const int64_t at = (((int64_t)s * n + (t - p0)) * c.H_kv + h) * 16 + 2 * g;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            uint32_t v[8];
            codes_to_f16(code[which][i].x, v[0], v[1], v[2], v[3]);
            codes_to_f16(code[which][i].y, v[4], v[5], v[6], v[7]);
            const uint32_t f = scale_f16x2(sc[which][i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = f16x2_to_bf16x2(mul_f16x2(v[e], f));
            store_once_32((which ? v_out : k_out) + at, v);
        }
    }
}

}  // namespace

int launch_append_kv4(const sba_cache4& c, const void* k_new, const void* v_new, const int32_t* pos_start, int n_new,
                      cudaStream_t stream) {
    dim3 grid((n_new - 1) / c.b + 2, c.H_kv, c.B);  // blocks a window of n_new positions can overlap
    return launch(c.b == 64 ? append_kv4_kernel<64> : append_kv4_kernel<128>, grid, dim3(kThreads), 0, stream, c,
                  reinterpret_cast<const uint4*>(k_new), reinterpret_cast<const uint4*>(v_new), pos_start, n_new);
}

int launch_read_kv4(const sba_cache4& c, const int32_t* pos_start, int n, void* k_out, void* v_out,
                    cudaStream_t stream) {
    dim3 grid((n - 1) / c.b + 2, c.H_kv, c.B);
    return launch(c.b == 64 ? read_kv4_kernel<64> : read_kv4_kernel<128>, grid, dim3(kThreads), 0, stream, c,
                  pos_start, n, reinterpret_cast<uint4*>(k_out), reinterpret_cast<uint4*>(v_out));
}

}  // namespace sba
