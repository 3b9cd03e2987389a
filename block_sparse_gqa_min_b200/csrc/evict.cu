// Eviction by accumulated attention weight: which tokens stay, and their rows moved to other pages.
//
// Per (sequence, KV head) the first n_sink and the last n_recent tokens stay, and of the rest the
// heaviest, up to n_keep in all (weight descending, then position ascending; -0 == +0, a NaN ranks
// below every number).  Kept tokens stay in order, so "recent" and the local blocks of later steps
// mean what they meant.  Two launches:
//  - evict_select_kernel: one thread-block cluster per (sequence, KV head).  The threshold is found by
//    a radix select, 8 bits of the order-preserving key a pass: every CTA histograms its slice of the
//    weights in shared memory, and all CTAs add the cluster's histograms through distributed shared
//    memory, so each pass is one cluster barrier.  The slice is read from L2 (or L1) again each pass:
//    4 bytes a token.  Two more passes count and write the kept positions, in order, without atomics.
//    It is bound by the latency of its dependent passes.
//  - gather kernels: one CTA per (destination block, KV head, sequence) moves the rows (whole rows,
//    16 bytes a lane, all loads of a thread issued before its first store), the accumulators, and forms the
//    block's Quest descriptor from the keys it holds in registers.  Bound by HBM.
#include <math.h>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.cuh"

namespace sba {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;  // the portable cluster size
constexpr int kMoveThreads = 256;

struct SelectArgs {
    const int32_t* seq_lens;
    const int32_t* block_table;
    int32_t* status;
    int H_kv, b, max_blocks, num_pages;
    const float* acc;
    sba_evict_params p;
    int32_t* kept;
    int32_t* new_lens;
};

__device__ __forceinline__ int clamped_len(const int32_t* seq_lens, int s, int max_blocks, int b) {
    return max(0, min(__ldca(seq_lens + s), max_blocks * b));
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(SelectArgs a) {
    __shared__ uint32_t hist[4][256];
    __shared__ uint32_t scan[8];
    __shared__ uint32_t found[2];  // digit of the threshold, tokens still to take at it
    __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
    __shared__ uint32_t totals[2];  // tokens of this CTA above and at the threshold

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y, s = blockIdx.z;
    const uint32_t rank = cluster_rank(), C = cluster_size();
    for (int i = tid; i < 4 * 256; i += kSelThreads) hist[i >> 8][i & 255] = 0;
    pdl_wait();
    pdl_trigger();
    const int n = clamped_len(a.seq_lens, s, a.max_blocks, a.b);
    const int keep = a.p.n_keep;
    int32_t* kept = a.kept + ((int64_t)s * a.H_kv + h) * keep;
    if (rank == 0 && h == 0 && tid == 0) a.new_lens[s] = min(n, keep);
    if (n <= keep) {
        for (int i = (int)rank * kSelThreads + tid; i < n; i += (int)C * kSelThreads) kept[i] = i;
        return;
    }
    const int sink = a.p.n_sink, recent = a.p.n_recent, k = keep - sink - recent;
    for (int i = (int)rank * kSelThreads + tid; i < sink; i += (int)C * kSelThreads) kept[i] = i;
    for (int i = (int)rank * kSelThreads + tid; i < recent; i += (int)C * kSelThreads)
        kept[keep - recent + i] = n - recent + i;
    if (k == 0) return;

    // this CTA's slice [lo, hi) of the ranked tokens, and this warp's part of it
    const int64_t m = n - recent - sink;
    const int lo = sink + (int)(m * rank / C), hi = sink + (int)(m * (rank + 1) / C);
    const int wlo = lo + (int)((int64_t)(hi - lo) * warp / kSelWarps);
    const int whi = lo + (int)((int64_t)(hi - lo) * (warp + 1) / kSelWarps);
    auto key_of = [&](int t) -> uint32_t {
        const int j = t / a.b;
        const int64_t page = page_of(a.block_table, a.max_blocks, a.num_pages, s, j, a.status);
        if (page < 0) return 0u;
        const float w = __ldca(a.acc + (page * a.H_kv + h) * a.b + (t - j * a.b));
        return w != w ? 0u : orderable_key(w);
    };

    __syncthreads();
    uint32_t prefix = 0, left = (uint32_t)k;  // left: tokens to take among those whose key starts with prefix
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int t0 = wlo; t0 < whi; t0 += 32) {
            const int t = t0 + lane;
            const uint32_t key = t < whi ? key_of(t) : 0u;
            const bool in = t < whi && (pass == 0 || (key >> (shift + 8)) == prefix);
            const uint32_t digit = in ? (key >> shift) & 255u : 256u;
            const uint32_t same = __match_any_sync(0xffffffffu, digit);
            if (in && (same & ((1u << lane) - 1u)) == 0) atomicAdd(&hist[pass][digit], (uint32_t)__popc(same));
        }
        cluster_sync();
        // digits from the top: thread d looks at digit 255 - d
        uint32_t c = 0, below = 0;
        if (tid < 256) {
            for (uint32_t r = 0; r < C; ++r) c += ld_peer_u32(peer_addr(&hist[pass][255 - tid], r));
            uint32_t sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (lane == 31) scan[warp] = sum;
            below = sum - c;
        }
        __syncthreads();
        if (tid < 256) {
            for (int w = 0; w < warp; ++w) below += scan[w];
            if (below < left && below + c >= left) {
                found[0] = 255 - tid;
                found[1] = left - below;
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | found[0];
        left = found[1];
        __syncthreads();
    }
    const uint32_t T = prefix;

    // tokens above and at the threshold: per warp, per CTA, then the CTAs before this one
    uint32_t gt = 0, eq = 0;
    for (int t0 = wlo; t0 < whi; t0 += 32) {
        const int t = t0 + lane;
        const uint32_t key = t < whi ? key_of(t) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, t < whi && key > T));
        eq += __popc(__ballot_sync(0xffffffffu, t < whi && key == T));
    }
    if (lane == 0) {
        warp_gt[warp] = gt;
        warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t g = 0, e = 0;
        for (int w = 0; w < kSelWarps; ++w) {
            const uint32_t gw = warp_gt[w], ew = warp_eq[w];
            warp_gt[w] = g;
            warp_eq[w] = e;
            g += gw;
            e += ew;
        }
        totals[0] = g;
        totals[1] = e;
    }
    cluster_sync();
    uint32_t g0 = warp_gt[warp], e0 = warp_eq[warp];
    for (uint32_t r = 0; r < rank; ++r) {
        g0 += ld_peer_u32(peer_addr(&totals[0], r));
        e0 += ld_peer_u32(peer_addr(&totals[1], r));
    }
    const uint32_t lower = (1u << lane) - 1u;
    for (int t0 = wlo; t0 < whi; t0 += 32) {
        const int t = t0 + lane;
        const uint32_t key = t < whi ? key_of(t) : 0u;
        const bool is_gt = t < whi && key > T, is_eq = t < whi && key == T;
        const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
        const uint32_t my_e = e0 + __popc(be & lower), my_g = g0 + __popc(bg & lower);
        if (is_gt || (is_eq && my_e < left)) kept[sink + my_g + min(my_e, left)] = t;
        g0 += __popc(bg);
        e0 += __popc(be);
    }
    cluster_sync();  // no CTA leaves while another still reads its shared memory
}

struct MoveArgs {
    const uint8_t* k_src;  // bf16 keys, or four-bit tiles
    const uint8_t* v_src;
    uint8_t* k_dst;
    uint8_t* v_dst;
    const float* acc_src;
    float* acc_dst;
    const int32_t* seq_lens;
    const int32_t* src_table;
    const int32_t* dst_table;
    int32_t* status;
    int32_t* dst_status;
    int H_kv, src_max_blocks, src_pages, dst_max_blocks, dst_pages, n_keep;
    const int32_t* kept;
    void* desc;
};

// Source rows (page, head, row) of this CTA's destination rows, -1 where none; returns their number.
template <int kBlk>
__device__ __forceinline__ int source_rows(const MoveArgs& a, int64_t* src, int64_t& dst_page) {
    const int jd = blockIdx.x, h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
    const int n = clamped_len(a.seq_lens, s, a.src_max_blocks, kBlk);
    const int rows = min(kBlk, min(n, a.n_keep) - jd * kBlk);
    if (rows <= 0) return 0;
    dst_page = page_of(a.dst_table, a.dst_max_blocks, a.dst_pages, s, jd, tid == 0 ? a.dst_status : nullptr);
    if (dst_page < 0) return 0;
    if (tid < kBlk) {
        int64_t from = -1;
        if (tid < rows) {
            const int t = __ldca(a.kept + ((int64_t)s * a.H_kv + h) * a.n_keep + jd * kBlk + tid);
            const int64_t page = page_of(a.src_table, a.src_max_blocks, a.src_pages, s, t / kBlk, a.status);
            if (page >= 0) from = (page * a.H_kv + h) * kBlk + t % kBlk;
        }
        src[tid] = from;
    }
    __syncthreads();
    if (a.acc_dst && tid < rows && src[tid] >= 0)
        a.acc_dst[(dst_page * a.H_kv + h) * kBlk + tid] = __ldca(a.acc_src + src[tid]);
    return rows;
}

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr uint32_t kInf2 = 0x7f807f80u, kNegInf2 = 0xff80ff80u;  // bf16x2

// bf16 cache: 16 lanes move a 256-byte row.
template <int kBlk>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(MoveArgs a) {
    constexpr int kIter = kBlk / 16;
    __shared__ int64_t src[kBlk];
    __shared__ uint32_t red[2][kMoveThreads / 32][64];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = tid & 15, r0 = tid >> 4;
    pdl_wait();
    pdl_trigger();
    int64_t page = -1;
    if (source_rows<kBlk>(a, src, page) == 0) return;
    const int64_t drow = (page * a.H_kv + blockIdx.y) * kBlk;
    uint32_t mn[4] = {kInf2, kInf2, kInf2, kInf2}, mx[4] = {kNegInf2, kNegInf2, kNegInf2, kNegInf2};
#pragma unroll
    for (int i0 = 0; i0 < kIter; i0 += 4) {
        uint4 k[4], v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t from = src[r0 + 16 * (i0 + i)];
            if (from >= 0) {
                k[i] = ld_once_v4(reinterpret_cast<const uint4*>(a.k_src) + from * 16 + c);
                v[i] = ld_once_v4(reinterpret_cast<const uint4*>(a.v_src) + from * 16 + c);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 16 * (i0 + i);
            if (src[r] < 0) continue;
            reinterpret_cast<uint4*>(a.k_dst)[(drow + r) * 16 + c] = k[i];
            reinterpret_cast<uint4*>(a.v_dst)[(drow + r) * 16 + c] = v[i];
            const uint32_t w[4] = {k[i].x, k[i].y, k[i].z, k[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mn[e] = min2(mn[e], w[e]);
                mx[e] = max2(mx[e], w[e]);
            }
        }
    }
    if (!a.desc) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        mn[e] = min2(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], 16));
        mx[e] = max2(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
        if (lane < 16) {
            red[0][warp][c * 4 + e] = mn[e];
            red[1][warp][c * 4 + e] = mx[e];
        }
    }
    __syncthreads();
    if (tid < 128) {
        const int which = tid >> 6, pair = tid & 63;
        uint32_t v = red[which][0][pair];
#pragma unroll
        for (int w = 1; w < kMoveThreads / 32; ++w) v = which ? max2(v, red[which][w][pair]) : min2(v, red[which][w][pair]);
        reinterpret_cast<uint32_t*>(a.desc)[((page * a.H_kv + blockIdx.y) * 2 + which) * 64 + pair] = v;
    }
}

// Four-bit cache: 8 lanes move a row, four for the key codes and four for the value codes (16 bytes each), every lane
// also two scales of its own 32 channels, so a key lane can form the descriptor from what it moves.
template <int kBlk>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kv4_kernel(MoveArgs a) {
    constexpr int kIter = kBlk / 32;
    __shared__ int64_t src[kBlk];
    __shared__ uint32_t red[2][kMoveThreads / 32][64];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = tid & 7, r = tid >> 3;
    pdl_wait();
    pdl_trigger();
    int64_t page = -1;
    if (source_rows<kBlk>(a, src, page) == 0) return;
    const int codes_at = (g < 4 ? 0 : kStripV) + (g & 3) * 16, scales_at = (g < 4 ? kStripKS : kStripVS) + (g & 3) * 2;
    uint8_t* tile = a.k_dst + (page * a.H_kv + blockIdx.y) * (int64_t)(kIter * kStripBytes);
    uint4 code[kIter];
    uint32_t sc[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int64_t from = src[r + 32 * i];
        if (from >= 0) {
            const uint8_t* strip = a.k_src + (from >> 5) * kStripBytes;
            code[i] = ld_once_v4(strip + (from & 31) * 64 + codes_at);
            sc[i] = __ldca(reinterpret_cast<const uint16_t*>(strip + (from & 31) * 8 + scales_at));
        }
    }
    __half2 mn[16], mx[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        mn[e] = __half2half2(__ushort_as_half(0x7c00));
        mx[e] = __half2half2(__ushort_as_half(0xfc00));
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        if (src[r + 32 * i] < 0) continue;
        uint8_t* strip = tile + i * kStripBytes;
        *reinterpret_cast<uint4*>(strip + r * 64 + codes_at) = code[i];
        *reinterpret_cast<uint16_t*>(strip + r * 8 + scales_at) = (uint16_t)sc[i];
        if (a.desc && g < 4) {
            const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t v[4];
                codes_to_f16(w[x], v[0], v[1], v[2], v[3]);
                const uint32_t f = scale_f16x2(x < 2 ? sc[i] & 0xffu : sc[i] >> 8);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t y = mul_f16x2(v[e], f);
                    mn[4 * x + e] = __hmin2(mn[4 * x + e], *reinterpret_cast<const __half2*>(&y));
                    mx[4 * x + e] = __hmax2(mx[4 * x + e], *reinterpret_cast<const __half2*>(&y));
                }
            }
        }
    }
    if (!a.desc) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            mn[e] = __hmin2(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], o));
            mx[e] = __hmax2(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
        }
        if (lane < 4) {
            red[0][warp][g * 16 + e] = f16x2_to_bf16x2(*reinterpret_cast<const uint32_t*>(&mn[e]));
            red[1][warp][g * 16 + e] = f16x2_to_bf16x2(*reinterpret_cast<const uint32_t*>(&mx[e]));
        }
    }
    __syncthreads();
    if (tid < 128) {
        const int which = tid >> 6, pair = tid & 63;
        uint32_t v = red[which][0][pair];
#pragma unroll
        for (int w = 1; w < kMoveThreads / 32; ++w) v = which ? max2(v, red[which][w][pair]) : min2(v, red[which][w][pair]);
        reinterpret_cast<uint32_t*>(a.desc)[((page * a.H_kv + blockIdx.y) * 2 + which) * 64 + pair] = v;
    }
}

// One cluster per (sequence, KV head): as many CTAs as fill the GPU, and as have 2048 tokens each.
int select_cluster(int64_t units, int max_len) {
    int C = 1;
    while (C < kMaxCluster && units * C * 2 <= 148 && max_len / (2 * C) >= 2048) C *= 2;
    return C;
}

template <class Cache>
int launch_select(const Cache& src, const float* acc, const sba_evict_params& p, int32_t* new_lens, int32_t* kept,
                  cudaStream_t stream) {
    SelectArgs a{src.seq_lens, src.block_table, src.status, src.H_kv, src.b, src.max_blocks, src.num_pages, acc, p, kept,
                 new_lens};
    const int C = select_cluster((int64_t)src.B * src.H_kv, src.max_len);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C, src.H_kv, src.B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
    if (e != cudaSuccess) {
        note_cuda_error(e);
        return SBA_ERR_CUDA;
    }
    return SBA_OK;
}

template <class Cache>
MoveArgs move_args(const Cache& src, const float* acc, const sba_evict_params& p, const Cache& dst, float* acc_dst,
                   const int32_t* kept) {
    MoveArgs m{};
    m.acc_src = acc;
    m.acc_dst = acc_dst;
    m.seq_lens = src.seq_lens;
    m.src_table = src.block_table;
    m.dst_table = dst.block_table;
    m.status = src.status;
    m.dst_status = dst.status;
    m.H_kv = src.H_kv;
    m.src_max_blocks = src.max_blocks;
    m.src_pages = src.num_pages;
    m.dst_max_blocks = dst.max_blocks;
    m.dst_pages = dst.num_pages;
    m.n_keep = p.n_keep;
    m.kept = kept;
    m.desc = dst.desc;
    return m;
}

}  // namespace

int launch_evict(const sba_cache& src, const float* acc, const sba_evict_params& p, const sba_cache& dst,
                 float* acc_dst, int32_t* new_lens, int32_t* kept, cudaStream_t stream) {
    const int rc = launch_select(src, acc, p, new_lens, kept, stream);
    if (rc != SBA_OK) return rc;
    MoveArgs m = move_args(src, acc, p, dst, acc_dst, kept);
    m.k_src = static_cast<const uint8_t*>(src.k);
    m.v_src = static_cast<const uint8_t*>(src.v);
    m.k_dst = static_cast<uint8_t*>(dst.k);
    m.v_dst = static_cast<uint8_t*>(dst.v);
    dim3 grid((p.n_keep + src.b - 1) / src.b, src.H_kv, src.B);
    return launch(src.b == 64 ? evict_move_kernel<64> : evict_move_kernel<128>, grid, dim3(kMoveThreads), 0, stream, m);
}

int launch_evict_kv4(const sba_cache4& src, const float* acc, const sba_evict_params& p, const sba_cache4& dst,
                     float* acc_dst, int32_t* new_lens, int32_t* kept, cudaStream_t stream) {
    const int rc = launch_select(src, acc, p, new_lens, kept, stream);
    if (rc != SBA_OK) return rc;
    MoveArgs m = move_args(src, acc, p, dst, acc_dst, kept);
    m.k_src = static_cast<const uint8_t*>(src.kv);
    m.k_dst = static_cast<uint8_t*>(dst.kv);
    dim3 grid((p.n_keep + src.b - 1) / src.b, src.H_kv, src.B);
    return launch(src.b == 64 ? evict_move_kv4_kernel<64> : evict_move_kv4_kernel<128>, grid, dim3(kMoveThreads), 0,
                  stream, m);
}

}  // namespace sba
