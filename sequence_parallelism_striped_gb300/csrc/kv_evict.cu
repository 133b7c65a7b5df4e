// kv_evict.cu -- which rows of a prompt stay in its cache, by the weight that
// attention gave them, and their move into a smaller one.
//
// Selection, one thread-block cluster per (sequence, key/value head): every
// weight becomes an unsigned number of the same order (kept in shared memory,
// in the order of the positions), the first `sinks` and last `recent`
// positions the largest number of all.  The keep-th largest number T is found
// digit by digit: a block counts the digits of its part, the cluster's
// blocks read one another's counts through distributed shared memory and each
// finds the same digit.  Above T all positions stay, of those at T the lowest
// ones; with the counts of the blocks before it every warp knows where its
// positions go, so the list is in order and nothing depends on timing.
//
// Bound by latency: a pass over the numbers and a cluster barrier per digit.  The
// move is bound by memory: kept rows are read and written once.  Measured, 8
// heads, 16384 of 131072 rows of 128 channels: 46 us, selection 24 (clusters of
// four blocks: 32, of sixteen: 63), move 22 (6.3 TB/s).
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace striped {

namespace {

constexpr int kEThreads = 1024;
constexpr int kEWarps = kEThreads / 32;
// 11, 11 and 10 bits: with 8 at a time, most weights of a prompt share a few first
// digits (an exponent less its last bit), and their counts are added one after
// another
constexpr int kDigitBits = 11;
constexpr int kDigit = 1 << kDigitBits;
constexpr int kBatch = 8;      // loads of a thread in flight
constexpr int kMaxBlocks = 8;  // of a cluster
// positions whose numbers a block holds in shared memory; a longer part is read
// from the weights (from L2) in every pass
constexpr int kEHeld = 49152;
constexpr int kGThreads = 256;
constexpr int kEPart = 8192;  // positions a block should have before a cluster gets a further one

struct Placement {
    int layout;  // contiguous: one stripe
    uint32_t N, S, L;
};
__device__ __forceinline__ uint32_t row_of(const Placement &g, uint32_t p) {
    if (g.N == 1) return p;
    if (g.layout == STRIPED_LAYOUT_STRIPED) return p % g.N * g.L + p / g.N;
    const uint32_t C = g.L / 2, c = p / C, in = p - c * C;
    return c < g.N ? c * g.L + in : (2 * g.N - 1 - c) * g.L + C + in;
}

// Same order as the weights; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

struct SelectArgs {
    const float *weight;  // [rows][S] in placed rows
    int32_t *index;       // [rows][keep]
    Placement g;
    uint32_t keep, sinks, recent;
    uint32_t part;        // positions of a block (a multiple of kEThreads)
};

struct SelectShared {
    uint32_t hist[2][kDigit];  // of this block, by the parity of the digit
    uint32_t above[kEWarps], at[kEWarps];
    uint32_t sum_above, sum_at;
    uint32_t digit, left;
};

__global__ void __launch_bounds__(kEThreads, 1) kv_select_kernel(const SelectArgs a) {
    extern __shared__ uint32_t held[];
    __shared__ SelectShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
    const int64_t line = blockIdx.x / blocks;
    const float *weight = a.weight + line * a.g.S;
    const uint32_t p0 = min(a.part * rank, a.g.S), p1 = min(p0 + a.part, a.g.S);
    const int n = (int)(p1 - p0);
    const bool hold = a.part <= kEHeld;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t tail = a.g.S - a.recent;
    auto number = [&](uint32_t p) -> uint32_t {
        if (p < a.sinks || p >= tail) return ~0u;
        return order_of(__ldg(weight + row_of(a.g, p)));
    };
    if (hold) {
        if (a.g.layout == STRIPED_LAYOUT_STRIPED && a.g.N > 1 && a.g.N <= 1024) {
            // stripe by stripe, so that neighbouring lanes read neighbouring rows
            const uint32_t N = a.g.N, per = n / N + 2, i0 = p0 / N;
            for (uint32_t f0 = threadIdx.x; f0 < per * N; f0 += kBatch * kEThreads) {
                uint32_t p[kBatch];
                float w[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const uint32_t f = f0 + k * kEThreads, d = f / per, i = i0 + (f - d * per);
                    p[k] = f < per * N ? i * N + d : 0xffffffffu;
                    w[k] = p[k] >= p0 && p[k] < p1 ? __ldg(weight + d * a.g.L + i) : 0.f;
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (p[k] >= p0 && p[k] < p1)
                        held[p[k] - p0] = p[k] < a.sinks || p[k] >= tail ? ~0u : order_of(w[k]);
            }
        } else {
            for (int i0 = threadIdx.x; i0 < n; i0 += kBatch * kEThreads) {
                uint32_t v[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) v[k] = i0 + k * kEThreads < n ? number(p0 + i0 + k * kEThreads) : 0u;
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (i0 + k * kEThreads < n) held[i0 + k * kEThreads] = v[k];
            }
        }
    }
    for (int i = threadIdx.x; i < 2 * kDigit; i += kEThreads) sh.hist[i / kDigit][i % kDigit] = 0;
    static_assert(kDigit == 2 * kEThreads && kEWarps == 32, "a thread has two digits, a lane a warp's sum");
    __syncthreads();
    // digits from the highest on; `left` of the numbers that begin with
    // `prefix` are among the largest `keep`
    uint32_t prefix = 0, left = a.keep;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int above_shift = pass == 1 ? 21 : 10;  // where the digits before this one end
        const uint32_t mask = pass == 2 ? 1023u : kDigit - 1u;
        uint32_t *hist = sh.hist[pass & 1];
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += kEThreads) {
            const uint32_t v = hold ? held[i] : number(p0 + i);
            if (pass == 0 || (v >> above_shift) == prefix) atomicAdd(&hist[(v >> shift) & mask], 1u);
        }
        cluster.sync();
        // thread t has the digits 2 t and 2 t + 1, over all blocks
        uint2 c = make_uint2(0u, 0u), part[kMaxBlocks];
#pragma unroll
        for (int b = 0; b < kMaxBlocks; ++b)
            part[b] = b < blocks ? reinterpret_cast<const uint2 *>(cluster.map_shared_rank(hist, b))[threadIdx.x]
                                 : make_uint2(0u, 0u);
#pragma unroll
        for (int b = 0; b < kMaxBlocks; ++b) c.x += part[b].x, c.y += part[b].y;
        // the counts of the other parity were read before this barrier
        reinterpret_cast<uint2 *>(sh.hist[(pass + 1) & 1])[threadIdx.x] = make_uint2(0u, 0u);
        // numbers of the higher digits: first those of this warp, then of others
        uint32_t run = c.x + c.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_down_sync(0xffffffffu, run, o);
            if (lane + o < 32) run += x;
        }
        if (lane == 0) sh.above[warp] = run;
        __syncthreads();
        uint32_t higher = sh.above[lane];  // lane w: what warp w has
        higher = __reduce_add_sync(0xffffffffu, lane > warp ? higher : 0u);
        uint32_t over = higher + run - (c.x + c.y);
        if (over < left && left <= over + c.y) sh.digit = 2 * threadIdx.x + 1, sh.left = left - over;
        over += c.y;
        if (over < left && left <= over + c.x) sh.digit = 2 * threadIdx.x, sh.left = left - over;
        __syncthreads();
        prefix = (prefix << (pass == 2 ? 10 : kDigitBits)) | sh.digit;
        left = sh.left;
    }
    // every warp counts a stretch of the block's positions, then writes it
    const int per = (int)(a.part / kEWarps);
    const int i0 = min(warp * per, n), i1 = min(i0 + per, n);
    uint32_t above = 0, at = 0;
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) {
        const uint32_t v = hold ? held[i] : number(p0 + i);
        above += v > prefix;
        at += v == prefix;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    at = __reduce_add_sync(0xffffffffu, at);
    if (lane == 0) sh.above[warp] = above, sh.at[warp] = at;
    __syncthreads();
    if (warp == 0) {
        const uint32_t sa = __reduce_add_sync(0xffffffffu, sh.above[lane]);
        const uint32_t st = __reduce_add_sync(0xffffffffu, sh.at[lane]);
        if (lane == 0) sh.sum_above = sa, sh.sum_at = st;
    }
    cluster.sync();
    uint32_t before_above = lane < warp ? sh.above[lane] : 0u, before_at = lane < warp ? sh.at[lane] : 0u;
    if (lane < rank) {
        before_above += *cluster.map_shared_rank(&sh.sum_above, lane);
        before_at += *cluster.map_shared_rank(&sh.sum_at, lane);
    }
    before_above = __reduce_add_sync(0xffffffffu, before_above);
    before_at = __reduce_add_sync(0xffffffffu, before_at);
    int32_t *index = a.index + line * a.keep;
#pragma unroll 4
    for (int i = i0; i < i1; i += 32) {
        const bool in = i + lane < i1;
        const uint32_t v = in ? (hold ? held[i + lane] : number(p0 + i + lane)) : 0u;
        const uint32_t up = __ballot_sync(0xffffffffu, in && v > prefix);
        const uint32_t eq = __ballot_sync(0xffffffffu, in && v == prefix);
        const uint32_t low = (1u << lane) - 1u;
        const uint32_t a0 = before_above + __popc(up & low), t0 = before_at + __popc(eq & low);
        const bool stays = (up >> lane & 1u) || ((eq >> lane & 1u) && t0 < left);
        if (stays) index[a0 + min(t0, left)] = (int32_t)(p0 + i + lane);
        before_above += __popc(up);
        before_at += __popc(eq);
    }
    cluster.sync();  // no block leaves while another may read its counts
}

// Rows of the call's tensors and the weights.
struct GatherArgs {
    const char *x[kEvictTensors + 1];
    char *y[kEvictTensors + 1];
    int row_bytes[kEvictTensors + 1];
    int lanes_log[kEvictTensors + 1];  // log2 of the lanes that move a row
    const int32_t *index;              // positions
    Placement g;
    uint32_t keep;
    int64_t lines;
};

// V a lane, 2^log lanes a row (more than a row has: some idle; fewer: they go on
// behind one another), two rows in flight: more take registers and with them
// lanes (16384 of 131072 rows, 8 heads: 42 us at 8 rows, 31 at 4, 22 so).
template <typename V>
__device__ __forceinline__ void gather_rows(const GatherArgs &a, int t) {
    const int log = a.lanes_log[t], per = a.row_bytes[t] / (int)sizeof(V);
    const uint32_t first = (blockIdx.x * kGThreads + threadIdx.x) >> log, step = (gridDim.x * kGThreads) >> log;
    const int c0 = threadIdx.x & ((1 << log) - 1);
    constexpr int U = 2;
    for (int64_t line = blockIdx.z; line < a.lines; line += gridDim.z) {
        const V *x = reinterpret_cast<const V *>(a.x[t]) + line * a.g.S * per;
        V *y = reinterpret_cast<V *>(a.y[t]) + line * a.keep * per;
        const int32_t *index = a.index + line * a.keep;
        for (uint32_t r = first; r < a.keep; r += U * step) {
            uint32_t from[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                from[k] = r + k * step < a.keep ? row_of(a.g, (uint32_t)index[r + k * step]) : 0u;
            for (int c = c0; c < per; c += 1 << log) {
                V v[U];
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if (r + k * step < a.keep) v[k] = __ldcs(x + (int64_t)from[k] * per + c);
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if (r + k * step < a.keep) __stcs(y + (int64_t)(r + k * step) * per + c, v[k]);
            }
        }
    }
}

__global__ void __launch_bounds__(kGThreads, 8) kv_gather_kernel(const GatherArgs a) {
    wait_for_previous();
    const int t = blockIdx.y;
    if (a.row_bytes[t] % 16 == 0) gather_rows<uint4>(a, t);
    else gather_rows<uint32_t>(a, t);
}

}  // namespace

int launch_kv_evict(const EvictArgs &e, cudaStream_t stream) {
    static PerDeviceOnce once;
    const int attr = once.get([] {
        return cuda_status(cudaFuncSetAttribute(kv_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                kEHeld * 4));
    });
    if (attr != STRIPED_OK) return attr;
    Placement g{};
    const bool one = e.layout == STRIPED_LAYOUT_CONTIGUOUS || e.N == 1;
    g.layout = one ? STRIPED_LAYOUT_STRIPED : e.layout;
    g.N = one ? 1u : (uint32_t)e.N;
    g.S = (uint32_t)e.S;
    g.L = g.S / g.N;
    SelectArgs s{};
    s.weight = e.weight;
    s.index = e.index;
    s.g = g;
    s.keep = (uint32_t)e.keep;
    s.sinks = (uint32_t)e.sinks;
    s.recent = (uint32_t)e.recent;
    int blocks = 1;
    while (blocks < kMaxBlocks && blocks * (int64_t)kEPart < e.S) blocks *= 2;
    s.part = (uint32_t)(((e.S + blocks - 1) / blocks + kEThreads - 1) / kEThreads * kEThreads);
    if (e.lines * blocks > 0x7fffffff) return STRIPED_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(e.lines * blocks));
    cfg.blockDim = dim3(kEThreads);
    cfg.dynamicSmemBytes = s.part <= kEHeld ? (size_t)s.part * 4 : 0;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)blocks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int st = cuda_status(cudaLaunchKernelEx(&cfg, kv_select_kernel, s));
    if (st) return st;
    GatherArgs ga{};
    uint64_t lanes = 1;  // of the tensor that has the most
    int n = 0;
    auto add = [&](const void *x, void *y, int64_t bytes) {
        ga.x[n] = static_cast<const char *>(x);
        ga.y[n] = static_cast<char *>(y);
        ga.row_bytes[n] = (int)bytes;
        const int64_t per = bytes / (bytes % 16 ? 4 : 16);
        int log = 0;
        while ((1 << log) < per && log < 5) ++log;
        ga.lanes_log[n++] = log;
        const uint64_t all = (uint64_t)e.keep << log;
        lanes = lanes > all ? lanes : all;
    };
    for (int i = 0; i < e.n; ++i) add(e.x[i], e.y[i], e.row_bytes[i]);
    if (e.weight_out) add(e.weight, e.weight_out, 4);
    ga.index = e.index;
    ga.g = g;
    ga.keep = s.keep;
    ga.lines = e.lines;
    if (n == 0) return STRIPED_OK;
    // two rows a lane, but no more blocks than fill the GPU a few times over
    const uint64_t z = e.lines < 65535 ? e.lines : 65535;
    uint64_t x = (lanes + 2 * kGThreads - 1) / (2 * kGThreads);
    const uint64_t most = (16 * (uint64_t)device_sm_count() + z - 1) / z;
    x = x > most ? most : x;
    return launch_after(kv_gather_kernel, dim3((unsigned)x, (unsigned)n, (unsigned)z), kGThreads, 0, stream, ga);
}

}  // namespace striped
