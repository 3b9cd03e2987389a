// Eviction by accumulated attention weight: which tokens stay, and their rows moved to other pages.
//
// Per (sequence, KV head) the first n_sink and the last n_recent tokens stay, and of the rest the
// heaviest, up to n_keep in all (weight descending, then position ascending; -0 == +0, a NaN ranks
// below every number).  Kept tokens stay in order, so "recent" and the local blocks of later steps
// mean what they meant.  Two launches:
//  - evict_select_kernel: one thread-block cluster per (sequence, KV head).  Every CTA reads its
//    slice of the weights once, four tokens a load, and keeps their order-preserving 32-bit keys in
//    shared memory (as far as they fit; the rest is read again from L2).  The threshold is found by a
//    radix select, 8 bits a pass: a shared-memory histogram of the slice, then one cluster barrier,
//    after which every CTA adds the cluster's histograms through distributed shared memory and finds
//    the same digit (256 bins: with 2048 and a pass less, reading ten peers' bins took 6 us a pass).  From the
//    second pass on a thread knows its tokens above the prefix and at it as bits and looks at the latter only;
//    once 1024 or fewer are left in the cluster, every CTA finds the last 16 bits alone.  An ordered write
//    follows; no position depends on an atomic.  64 units of 32-64K tokens: 20 us, 8 units of 512K: 25 us
//    (reading and counting 9, the second pass 5, the last digits 5, the write 3.5, barriers and digits the
//    rest): it is bound by the instructions of the first two passes (10 CTAs a unit: 13 quads a thread) and the
//    latency of what follows.
//  - gather kernels: one CTA per (destination block, KV head, sequence) moves the rows (whole rows,
//    16 bytes a lane, all loads of a thread issued before its first store), the accumulators, and forms
//    the block's Quest descriptor from the keys it holds in registers.  262144 bf16 rows: 48 us, 5.6 TB/s
//    read and written; as many four-bit rows: 26 us (a kept row's 144 bytes lie in four pieces that cost 256
//    bytes of DRAM access).
#include <math.h>

#include <mutex>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.cuh"

namespace sba {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBins = 256;
constexpr int kCopies = 8;                  // of the first histogram, by lane: most weights share few exponents
constexpr int kCopyStride = kBins + 4;      // words: the copies of a bin in different banks
constexpr int kSelFixed = (kCopies * kCopyStride + 3 * kBins) * 4;
constexpr int kSelMaxKeys = (226 * 1024 - kSelFixed) / 16 * 4;  // keys of a slice kept in shared memory
static_assert(kSelMaxKeys <= 15 * 4 * kSelThreads, "a thread's run of held keys has a bit each");
constexpr int kMoveThreads = 256;

struct SelectArgs {
    const int32_t* seq_lens;
    const int32_t* block_table;
    int32_t* status;
    int H_kv, b, log2_b, max_blocks, num_pages;
    const float* acc;
    sba_evict_params p;
    int32_t* kept;
    int32_t* new_lens;
};

__device__ __forceinline__ int clamped_len(const int32_t* seq_lens, int s, int max_blocks, int b) {
    return max(0, min(__ldca(seq_lens + s), max_blocks * b));
}

// Larger for a larger weight, the same for both zeros; 1 for a NaN.
__device__ __forceinline__ uint32_t key_of(float w) {
    return w != w ? 1u : orderable_key(w);
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(SelectArgs a, int cap) {
    extern __shared__ __align__(16) uint32_t dyn[];
    uint32_t* keys = dyn + kSelFixed / 4;
    __shared__ uint32_t scan[kSelWarps];
    __shared__ uint32_t found[3];  // digit of the threshold, tokens still to take at it, tokens that share it
    __shared__ uint32_t listed;    // tokens of this CTA in the list of the last two digits
    __shared__ uint2 warp_n[kSelWarps];
    __shared__ uint2 total;  // tokens of this CTA above and at the threshold

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y, s = blockIdx.z;
    const uint32_t rank = cluster_rank(), C = cluster_size();
    for (int i = tid; i < kSelFixed / 4; i += kSelThreads) dyn[i] = 0;
    if (tid == 0) listed = 0;
    pdl_wait();
    const int n = clamped_len(a.seq_lens, s, a.max_blocks, a.b);
    const int keep = a.p.n_keep;
    int32_t* kept = a.kept + ((int64_t)s * a.H_kv + h) * keep;
    if (rank == 0 && h == 0 && tid == 0) a.new_lens[s] = min(n, keep);
    if (n <= keep) {
        for (int i = (int)rank * kSelThreads + tid; i < n; i += (int)C * kSelThreads) kept[i] = i;
        return;
    }
    const int sink = a.p.n_sink, last = n - a.p.n_recent, k = keep - sink - a.p.n_recent;  // ranked: [sink, last)
    for (int i = (int)rank * kSelThreads + tid; i < sink; i += (int)C * kSelThreads) kept[i] = i;
    for (int i = (int)rank * kSelThreads + tid; i < n - last; i += (int)C * kSelThreads)
        kept[keep - (n - last) + i] = last + i;
    if (k == 0) return;

    // this CTA's slice: quads of tokens [q0, q0 + nq)
    const int n4 = (n + 3) / 4;
    const int q0 = (int)((int64_t)n4 * rank / C), nq = (int)((int64_t)n4 * (rank + 1) / C) - q0;
    // where quad i's weights are (cells fit 32 bits: a cache has fewer than 2^31 rows), -1 on a bad page
    auto cell_of = [&](int i) -> int {
        const int t = 4 * (q0 + i), j = t >> a.log2_b;
        const int page = a.block_table ? __ldca(a.block_table + (int64_t)s * a.max_blocks + j) : s * a.max_blocks + j;
        return page >= 0 && page < a.num_pages ? (page * a.H_kv + h) * a.b + (t & (a.b - 1)) : -1;
    };
    auto weights_of = [&](int cell) {  // a bad page's tokens rank last
        return cell >= 0 ? __ldca(reinterpret_cast<const float4*>(a.acc + cell)) : make_float4(NAN, NAN, NAN, NAN);
    };
    // keys of quad i: 0 outside the ranked tokens, 1 for a NaN, larger for a larger weight
    auto keys_of = [&](int i, float4 w) {
        const int t = 4 * (q0 + i);
        uint4 r;
        r.x = key_of(w.x);
        r.y = key_of(w.y);
        r.z = key_of(w.z);
        r.w = key_of(w.w);
        if (t < sink || t + 3 >= last) {
            if (t < sink || t >= last) r.x = 0;
            if (t + 1 < sink || t + 1 >= last) r.y = 0;
            if (t + 2 < sink || t + 2 >= last) r.z = 0;
            if (t + 3 < sink || t + 3 >= last) r.w = 0;
        }
        return r;
    };
    auto quad = [&](int i) -> uint4 {
        return 4 * i < cap ? *reinterpret_cast<const uint4*>(keys + 4 * i) : keys_of(i, weights_of(cell_of(i)));
    };

    __syncthreads();
    // ---- read the slice; histogram of the top 8 bits.  Asynchronous copies (what little L1 the keys leave could
    // not hold this many loads in flight), kLoads quads a thread at a time: one batch is counted while the next
    // is copied and the pages of the one after are looked up ----
    uint32_t* own = dyn + (lane & (kCopies - 1)) * kCopyStride;
    auto count = [&](uint4 r) {  // tokens that are not ranked too: in the last bin, whose number decides nothing
        atomicAdd(&own[r.x >> 24], 1u);
        atomicAdd(&own[r.y >> 24], 1u);
        atomicAdd(&own[r.z >> 24], 1u);
        atomicAdd(&own[r.w >> 24], 1u);
    };
    const int held = min(nq, cap / 4);
    constexpr int kLoads = 2, kStep = kLoads * kSelThreads;
    int cell[kLoads];
    auto look_up = [&](int i) {
#pragma unroll
        for (int x = 0; x < kLoads; ++x) cell[x] = i + x * kSelThreads < held ? cell_of(i + x * kSelThreads) : 0;
    };
    auto copy = [&](int i) {
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            uint32_t* to = keys + 4 * (i + x * kSelThreads);
            if (i + x * kSelThreads >= held) break;
            if (cell[x] >= 0) {
                cp_async_16(to, a.acc + cell[x]);
            } else {
                report(a.status, SBA_DEV_BAD_PAGE);
                *reinterpret_cast<float4*>(to) = weights_of(-1);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(tid);
    copy(tid);
    look_up(tid + kStep);
    for (int b0 = tid; b0 < held; b0 += kStep) {
        copy(b0 + kStep);
        look_up(b0 + 2 * kStep);
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // this thread's own, and it reads no other's
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            const int i = b0 + x * kSelThreads;
            if (i >= held) break;
            const uint4 r = keys_of(i, *reinterpret_cast<const float4*>(keys + 4 * i));
            *reinterpret_cast<uint4*>(keys + 4 * i) = r;
            count(r);
        }
    }
#pragma unroll 2
    for (int i = tid + (held - tid + kSelThreads - 1) / kSelThreads * kSelThreads; i < nq; i += kSelThreads) {
        const int at = cell_of(i);
        if (at < 0) report(a.status, SBA_DEV_BAD_PAGE);  // here once; the later passes look at it again
        count(keys_of(i, weights_of(at)));
    }
    __syncthreads();
    if (tid < kBins) {
        uint32_t c = 0;
#pragma unroll
        for (int x = 0; x < kCopies; ++x) c += dyn[x * kCopyStride + tid];
        dyn[tid] = c;
    }
    uint32_t prefix = 0, left = (uint32_t)k;  // left: tokens to take among those whose key starts with prefix
    // Runs: where all keys are held, a thread keeps in two masks which tokens of its own run of quads (an odd
    // number of them: its 16-byte reads then fall in different banks) are above the prefix and which are at it,
    // so that after the second pass only those at it are looked at again.
    const bool runs = 4 * nq <= cap;
    const int per = ((nq + kSelThreads - 1) / kSelThreads) | 1;
    const int i0 = min(nq, tid * per), i1 = min(nq, i0 + per);
    uint32_t above[2] = {0, 0}, at[2] = {0, 0};
    auto sift = [&](uint32_t top, int shift, auto same) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
            for (uint32_t rest = at[y]; rest; rest &= rest - 1) {
                const int bit = __ffs(rest) - 1;
                const uint32_t v = keys[4 * i0 + 32 * y + bit], u = v >> shift;
                if (u == top) {
                    same(v);
                } else {
                    at[y] ^= 1u << bit;
                    if (u > top) above[y] |= 1u << bit;
                }
            }
    };
    bool few = false;                         // every thread of every CTA holds at most one of them: low_key
    uint32_t low_key = ~0u;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        uint32_t* hist = pass == 0 ? dyn : dyn + kCopies * kCopyStride + (pass - 1) * kBins;
        const int shift = 24 - 8 * pass;
        if (few) {
            if (low_key >> (shift + 8) == (prefix & (0xffffu >> (shift + 8)))) atomicAdd(&hist[(low_key >> shift) & 255u], 1u);
        } else if (pass == 1 && runs) {
            const uint32_t lo = max(1u, prefix << 24), hi = prefix << 24 | 0xffffffu;
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                    const int i = i0 + 8 * y + z;
                    if (i >= i1) break;
                    const uint4 r = *reinterpret_cast<const uint4*>(keys + 4 * i);
                    const uint32_t v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        if (v[x] > hi) above[y] |= 1u << (4 * z + x);
                        if (v[x] - lo <= hi - lo) {
                            at[y] |= 1u << (4 * z + x);
                            atomicAdd(&hist[(v[x] >> 16) & 255u], 1u);
                        }
                    }
                }
        } else if (pass > 1 && runs) {
            sift(prefix, shift + 8, [&](uint32_t v) { atomicAdd(&hist[(v >> shift) & 255u], 1u); });
        } else if (pass > 0) {
#pragma unroll 4
            for (int i = tid; i < nq; i += kSelThreads) {
                const uint4 r = quad(i);
                if (r.x >> (shift + 8) == prefix && r.x) atomicAdd(&hist[(r.x >> shift) & 255u], 1u);
                if (r.y >> (shift + 8) == prefix && r.y) atomicAdd(&hist[(r.y >> shift) & 255u], 1u);
                if (r.z >> (shift + 8) == prefix && r.z) atomicAdd(&hist[(r.z >> shift) & 255u], 1u);
                if (r.w >> (shift + 8) == prefix && r.w) atomicAdd(&hist[(r.w >> shift) & 255u], 1u);
            }
        }
        if (few)
            __syncthreads();
        else
            cluster_sync();
        // digits from the top: thread d of the first eight warps takes bin 255 - d
        uint32_t mine = 0, sum = 0;
        if (tid < kBins) {
            if (few) {
                mine = hist[kBins - 1 - tid];
            } else {
                uint32_t c[kMaxCluster];  // all loads before the first sum
#pragma unroll
                for (uint32_t r = 0; r < kMaxCluster; ++r) c[r] = r < C ? ld_peer_u32(peer_addr(&hist[kBins - 1 - tid], r)) : 0u;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) mine += c[r];
            }
            sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (lane == 31) scan[warp] = sum;
        }
        __syncthreads();
        if (tid < kBins) {
            uint32_t before = sum - mine;  // tokens in higher bins
#pragma unroll
            for (int w = 0; w < kBins / 32; ++w)
                if (w < warp) before += scan[w];
            if (before < left && before + mine >= left) {
                found[0] = kBins - 1 - tid;
                found[1] = left - before;
                found[2] = mine;
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | found[0];
        left = found[1];
        if (pass == 1 && found[2] <= kSelThreads) {
            // The tokens that share the threshold's upper 16 bits have a thread each: every CTA lists its own
            // (where the first histogram was: the peers have read it), then takes one of all of them, and the
            // last two digits need no other CTA.
            few = true;
            auto list = [&](uint32_t v) {
                const uint32_t to = atomicAdd(&listed, 1u);
                if (to < kSelThreads) dyn[to] = v & 0xffffu;
            };
            if (runs) {
                sift(prefix, 16, list);
            } else {
#pragma unroll 4
                for (int i = tid; i < nq; i += kSelThreads) {
                    const uint4 r = quad(i);
                    if (r.x >> 16 == prefix && r.x) list(r.x);
                    if (r.y >> 16 == prefix && r.y) list(r.y);
                    if (r.z >> 16 == prefix && r.z) list(r.z);
                    if (r.w >> 16 == prefix && r.w) list(r.w);
                }
            }
            cluster_sync();
            const uint32_t theirs = lane < C ? ld_peer_u32(peer_addr(&listed, lane)) : 0u;
            uint32_t upto = theirs;
#pragma unroll
            for (int o = 1; o < kMaxCluster; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            uint32_t owner = 0, from = 0;  // the last CTA whose list starts at or before this thread
            for (uint32_t r = 1; r < C; ++r) {
                const uint32_t at = __shfl_sync(0xffffffffu, upto, r - 1);
                if ((uint32_t)tid >= at) {
                    owner = r;
                    from = at;
                }
            }
            if ((uint32_t)tid < __shfl_sync(0xffffffffu, upto, C - 1)) low_key = ld_peer_u32(peer_addr(&dyn[tid - from], owner));
        }
        __syncthreads();
    }
    const uint32_t T = prefix;

    // ---- tokens above and at the threshold, in order: every thread has a run of quads, so that nothing has to
    // be counted across lanes but the threads' totals ----
    uint32_t gt = 0, eq = 0;
    if (runs) {
        sift(T, 0, [](uint32_t) {});
        gt = __popc(above[0]) + __popc(above[1]);
        eq = __popc(at[0]) + __popc(at[1]);
    } else {
#pragma unroll 4
        for (int i = i0; i < i1; ++i) {
            const uint4 r = quad(i);
            gt += (r.x > T) + (r.y > T) + (r.z > T) + (r.w > T);
            eq += (r.x == T) + (r.y == T) + (r.z == T) + (r.w == T);
        }
    }
    uint32_t g = gt, e = eq;  // the tokens of this thread and those before it: warp, CTA, cluster
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t vg = __shfl_up_sync(0xffffffffu, g, o), ve = __shfl_up_sync(0xffffffffu, e, o);
        if (lane >= o) {
            g += vg;
            e += ve;
        }
    }
    if (lane == 31) warp_n[warp] = make_uint2(g, e);
    __syncthreads();
    const uint2 n_w = lane < warp ? warp_n[lane] : make_uint2(0u, 0u);
    g += __reduce_add_sync(0xffffffffu, n_w.x) - gt;
    e += __reduce_add_sync(0xffffffffu, n_w.y) - eq;
    if (tid == kSelThreads - 1) total = make_uint2(g + gt, e + eq);
    cluster_sync();
    uint2 n_c = make_uint2(0u, 0u);
    if (lane < rank) {
        n_c.x = ld_peer_u32(peer_addr(&total.x, lane));
        n_c.y = ld_peer_u32(peer_addr(&total.y, lane));
    }
    g += __reduce_add_sync(0xffffffffu, n_c.x);
    e += __reduce_add_sync(0xffffffffu, n_c.y);
    pdl_trigger();
    if (runs) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
            for (uint32_t rest = above[y] | at[y]; rest; rest &= rest - 1) {
                const int bit = __ffs(rest) - 1;
                const bool is_at = at[y] >> bit & 1;
                if (!is_at || e < left) kept[sink + g + min(e, left)] = 4 * (q0 + i0) + 32 * y + bit;
                g += !is_at;
                e += is_at;
            }
    } else if (gt + eq > 0) {
        for (int i = i0; i < i1; ++i) {
            const uint4 r = quad(i);
            const uint32_t v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (v[x] < T) continue;
                // (keys that are read again could have changed: nothing is written past the row)
                if ((v[x] > T || e < left) && sink + g + min(e, left) < keep) kept[sink + g + min(e, left)] = 4 * (q0 + i) + x;
                g += v[x] > T;
                e += v[x] == T;
            }
        }
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
    // the position, the length and the destination page do not wait for one another
    const bool in = tid < kBlk && jd * kBlk + tid < a.n_keep;
    const int t = in ? __ldca(a.kept + ((int64_t)s * a.H_kv + h) * a.n_keep + jd * kBlk + tid) : 0;
    dst_page = page_of(a.dst_table, a.dst_max_blocks, a.dst_pages, s, jd, nullptr);
    const int n = clamped_len(a.seq_lens, s, a.src_max_blocks, kBlk);
    const int rows = min(kBlk, min(n, a.n_keep) - jd * kBlk);
    if (rows <= 0) return 0;
    if (dst_page < 0) {
        if (tid == 0) report(a.dst_status, SBA_DEV_BAD_PAGE);
        return 0;
    }
    if (tid < kBlk) {
        int64_t from = -1;
        if (tid < rows) {
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

// Four-bit cache: 8 lanes move a row, four for the key codes and four for the value codes (16 bytes
// each), every lane also the two scales of its own 32 channels.  For the descriptor the value lanes
// take the upper half of a key lane's channels: 16 channels a lane keep the registers few, so that
// many CTAs share an SM (the kernel waits for its dependent loads, not for bandwidth); the threads'
// minima and maxima meet in shared memory.
constexpr int kMove4Threads = 128;
template <int kBlk>
__global__ void __launch_bounds__(kMove4Threads, kBlk == 64 ? 12 : 8) evict_move_kv4_kernel(MoveArgs a) {
    constexpr int kRowsAt = kMove4Threads / 8, kIter = kBlk / kRowsAt;
    __shared__ int64_t src[kBlk];
    __shared__ __half2 red[2][64][kRowsAt + 1];
    const int tid = threadIdx.x, lane = tid & 31, g = tid & 7, r = tid >> 3;
    pdl_trigger();
    int64_t page = -1;
    if (source_rows<kBlk>(a, src, page) == 0) return;
    const int codes_at = (g < 4 ? 0 : kStripV) + (g & 3) * 16, scales_at = (g < 4 ? kStripKS : kStripVS) + (g & 3) * 2;
    uint8_t* tile = a.k_dst + (page * a.H_kv + blockIdx.y) * (int64_t)(kBlk / kStripTokens * kStripBytes);
    uint4 code[kIter];
    uint32_t sc[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int64_t from = src[r + kRowsAt * i];
        code[i] = make_uint4(0u, 0u, 0u, 0u);
        sc[i] = 0;
        if (from >= 0) {
            const uint8_t* strip = a.k_src + (from >> 5) * kStripBytes;
            code[i] = ld_once_v4(strip + (from & 31) * 64 + codes_at);
            sc[i] = __ldca(reinterpret_cast<const uint16_t*>(strip + (from & 31) * 8 + scales_at));
        }
    }
    __half2 mn[8], mx[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        mn[e] = __half2half2(__ushort_as_half(0x7c00));
        mx[e] = __half2half2(__ushort_as_half(0xfc00));
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int row = r + kRowsAt * i;
        const bool real = src[row] >= 0;
        if (real) {
            uint8_t* strip = tile + (row >> 5) * kStripBytes;
            *reinterpret_cast<uint4*>(strip + (row & 31) * 64 + codes_at) = code[i];
            *reinterpret_cast<uint16_t*>(strip + (row & 31) * 8 + scales_at) = (uint16_t)sc[i];
        }
        if (a.desc) {  // channels 32(g % 4) + 16(g / 4) ..: the key lane's words x, y or z, w
            const uint32_t z = __shfl_sync(0xffffffffu, code[i].z, lane & ~4), w = __shfl_sync(0xffffffffu, code[i].w, lane & ~4);
            const uint32_t ks = __shfl_sync(0xffffffffu, sc[i], lane & ~4);
            uint32_t v[8];
            codes_to_f16(g < 4 ? code[i].x : z, v[0], v[1], v[2], v[3]);
            codes_to_f16(g < 4 ? code[i].y : w, v[4], v[5], v[6], v[7]);
            // a row that is not there counts as a NaN, which minimum and maximum pass over
            const uint32_t f = scale_f16x2(!real ? kScaleNaN : g < 4 ? ks & 0xffu : ks >> 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t y = mul_f16x2(v[e], f);
                mn[e] = __hmin2(mn[e], *reinterpret_cast<const __half2*>(&y));
                mx[e] = __hmax2(mx[e], *reinterpret_cast<const __half2*>(&y));
            }
        }
    }
    if (!a.desc) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int pair = (g & 3) * 16 + (g >> 2) * 8 + e;
        red[0][pair][r] = mn[e];
        red[1][pair][r] = mx[e];
    }
    __syncthreads();
    const int which = tid >> 6, pair = tid & 63;
    __half2 v = red[which][pair][0];
#pragma unroll
    for (int i = 1; i < kRowsAt; ++i) v = which ? __hmax2(v, red[which][pair][i]) : __hmin2(v, red[which][pair][i]);
    reinterpret_cast<uint32_t*>(a.desc)[((page * a.H_kv + blockIdx.y) * 2 + which) * 64 + pair] =
        f16x2_to_bf16x2(*reinterpret_cast<const uint32_t*>(&v));
}

cudaLaunchConfig_t select_config(int C, int H_kv, int B, int smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C, H_kv, B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cfg;
}

// Clusters of C CTAs (one CTA per SM) that the current device keeps resident at once; asked once per
// device and size.
int resident_clusters(int C) {
    static std::mutex lock;
    static int known[64][kMaxCluster + 1] = {};  // answer + 1
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> hold(lock);
    if (known[dev][0] == 0) {
        if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return 0;
        known[dev][0] = 1;
    }
    if (known[dev][C] == 0) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = select_config(C, 1, 1, kSelFixed + kSelMaxKeys * 4, nullptr, attr);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, evict_select_kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        known[dev][C] = n + 1;
    }
    return known[dev][C] - 1;
}

// CTAs per (sequence, KV head): the most whose clusters are all resident at once, with 4096 tokens a
// CTA at least (a smaller slice costs less than the larger cluster's barriers); one if the units
// alone fill the GPU.
int select_cluster(int64_t units, int max_len) {
    int most = max_len / 4096;
    if (most > kMaxCluster) most = kMaxCluster;
    for (int C = most; C > 1; --C)
        if (units * C <= 148 && resident_clusters(C) >= units) return C;
    return 1;
}

template <class Cache>
int launch_select(const Cache& src, const float* acc, const sba_evict_params& p, int32_t* new_lens, int32_t* kept,
                  cudaStream_t stream) {
    SelectArgs a{src.seq_lens, src.block_table, src.status, src.H_kv, src.b, src.b == 64 ? 6 : 7, src.max_blocks, src.num_pages, acc, p, kept,
                 new_lens};
    if (allow_smem<evict_select_kernel>(kSelFixed + kSelMaxKeys * 4) != SBA_OK) return SBA_ERR_CUDA;
    const int C = select_cluster((int64_t)src.B * src.H_kv, src.max_len);
    const int64_t slice = (((int64_t)src.max_len + 3) / 4 + C - 1) / C * 4;
    const int cap = (int)(slice < kSelMaxKeys ? slice : kSelMaxKeys);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = select_config(C, src.H_kv, src.B, kSelFixed + cap * 4, stream, attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cap);
    if (e != cudaSuccess) {
        note_cuda_error(e);
        return SBA_ERR_CUDA;
    }
    return SBA_OK;
}

// In plain stream order: launched early, its CTAs waited on the SMs that the selection left idle, and
// evict_512k took 71 us instead of 66.  (The kernel after it may start early: that is its own launch's attribute.)
int launch_move(void (*kernel)(MoveArgs), dim3 grid, int threads, const MoveArgs& m, cudaStream_t stream) {
    kernel<<<grid, threads, 0, stream>>>(m);
    return SBA_OK;  // the caller looks at cudaGetLastError
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
    return launch_move(src.b == 64 ? evict_move_kernel<64> : evict_move_kernel<128>, grid, kMoveThreads, m, stream);
}

int launch_evict_kv4(const sba_cache4& src, const float* acc, const sba_evict_params& p, const sba_cache4& dst,
                     float* acc_dst, int32_t* new_lens, int32_t* kept, cudaStream_t stream) {
    const int rc = launch_select(src, acc, p, new_lens, kept, stream);
    if (rc != SBA_OK) return rc;
    MoveArgs m = move_args(src, acc, p, dst, acc_dst, kept);
    m.k_src = static_cast<const uint8_t*>(src.kv);
    m.k_dst = static_cast<uint8_t*>(dst.kv);
    dim3 grid((p.n_keep + src.b - 1) / src.b, src.H_kv, src.B);
    return launch_move(src.b == 64 ? evict_move_kv4_kernel<64> : evict_move_kv4_kernel<128>, grid, kMove4Threads, m,
                       stream);
}

}  // namespace sba
