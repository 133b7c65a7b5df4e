// attn_window_fwd.cu -- bf16 causal attention over a sliding window and a few
// first tokens (sinks), forward, on tcgen05.
//
// Query position p keeps key position t iff t <= p and (p - t < W or
// t < sinks); the placement of the rows is that of the full attention
// (research.elamur.ai summary page, §Summary "every N-th token").  Tiles are
// 128 (or N * (128 / N)) consecutive positions, see window.cuh; query tile a
// visits the sink tiles 0 .. and the tiles from its window's lower edge to
// its own.
//
// One CTA = query tiles A = 2u and B = 2u + 1 of one head on one K/V stream:
// their windows differ by one tile.  The K/V tiles of the pair are
//   [0, ns) (sink tiles below the window), [lo(A), B];
// group A takes all but the last (key tile B lies after it), group B all but
// tile lo(A) when that is below its own window and holds no sink.
//   warp 0      TMA producer: Q_A, Q_B once, then K/V tiles
//   warp 1      TMEM allocator + single-thread tcgen05.mma issuer
//   warps 2..5  softmax group A, thread t owns query row t
//   warps 6..9  softmax group B
// Tensor memory: S_A [0,128), S_B [128,256), O_A [256,256+HD), O_B
// [384,384+HD); P is written back over S as bf16 pairs, the A operand of
// O += P V.  The running max moves lazily (by more than 2^8), which is exact
// because the final division uses the same reference.  P is rounded to bf16
// as a tensor-core operand; the row sum adds the unrounded values.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "window.cuh"

namespace striped {

namespace {

constexpr int WB = 128;                 // tile edge
constexpr uint32_t kWBox = 128 * 128;   // 128 rows x 64 bf16
constexpr int kWMaxNS = 4;
constexpr int kWThreads = 320;
constexpr float kWRescale = 8.0f;       // lazy rescale threshold, log2 units

template <int HD>
struct WinCfg {
    static constexpr int NS = HD == 128 ? 2 : 4;  // K/V stages
    static constexpr uint32_t kTile = (HD / 64) * kWBox;
    static constexpr uint32_t kQOff = 0;  // Q_A, then Q_B
    static constexpr uint32_t kKVOff = 2 * kTile;
    static constexpr uint32_t kStage = 2 * kTile;
    static constexpr uint32_t kPosOff = kKVOff + NS * kStage;  // position of every column of a tile
    static constexpr uint32_t kBarOff = kPosOff + WB * 4;
    static constexpr size_t kSmemBytes = 1024 + kBarOff + 256;
    static_assert(kSmemBytes <= 232448, "shared memory over the per-block limit");
    static_assert(NS <= kWMaxNS, "barrier array");
};

struct WinBars {
    uint64_t q_full;
    uint64_t kv_full[kWMaxNS], kv_empty[kWMaxNS];
    uint64_t s_full[2], p_ready[2], o_done[2];  // per softmax group
    uint64_t drain;                             // every MMA of the issuer has completed
    uint32_t tmem_slot;
};

struct WinParams {
    PosGeom g;
    int W, sinks;
    int nst;      // sink tiles
    int npair;    // query tile pairs of a head
    int G;        // query heads per key/value head
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    WaitCtl wc;
};

template <int HD>
__global__ void __launch_bounds__(kWThreads, 1)
    tc_window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const WinParams p) {
    using Cfg = WinCfg<HD>;
    constexpr int NS = Cfg::NS;
    constexpr uint32_t kTile = Cfg::kTile, kQOff = Cfg::kQOff, kKVOff = Cfg::kKVOff, kStage = Cfg::kStage;
    constexpr int kBoxes = HD / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    WinBars *bars = reinterpret_cast<WinBars *>(smem + Cfg::kBarOff);
    int *col_pos = reinterpret_cast<int *>(smem + Cfg::kPosOff);
    const uint32_t sbase = smem_u32(smem);
    const PosGeom &g = p.g;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    // head-major order: resident CTAs share the K/V tiles of one head in L2
    const int64_t bh = blockIdx.x / p.npair;
    const int u = blockIdx.x % p.npair;
    const int qa = 2 * u, qb = 2 * u + 1;
    const bool has_b = qb < g.nt;
    const int lo_a = window_lo(g, qa, p.W), lo_b = window_lo(g, qb, p.W);
    const int ns = min(p.nst, lo_a);
    const int nt = ns + (has_b ? qb : qa) - lo_a + 1;  // K/V tiles of the pair
    // group A: [0, n_a); group B: [0, nt) without `skip`
    const int n_a = has_b ? nt - 1 : nt;
    const int skip = (lo_b > lo_a && lo_a >= p.nst) ? ns : -1;
    const int kvh = (int)(bh / p.G);

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), 1);
            mbar_init(smem_u32(&bars->kv_empty[s]), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&bars->s_full[x]), 1);
            mbar_init(smem_u32(&bars->p_ready[x]), 4);
            mbar_init(smem_u32(&bars->o_done[x]), 1);
        }
        mbar_init(smem_u32(&bars->drain), 1);
        fence_barrier_init();
    }
    if (threadIdx.x < WB) col_pos[threadIdx.x] = threadIdx.x < g.P ? tile_pos(g, threadIdx.x) : 0x3fffffff;
    if (g.P < WB) {
        // rows past the tile's positions are never loaded: they must hold
        // finite values, because P = 0 times them is added to O
        for (uint32_t i = threadIdx.x * 16; i < kKVOff + NS * kStage; i += kWThreads * 16)
            *reinterpret_cast<uint4 *>(smem + i) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_slot;

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        const uint32_t box_bytes = (uint32_t)g.P * 128;
        const uint32_t qbar = smem_u32(&bars->q_full);
        mbar_arrive_expect_tx(qbar, (has_b ? 2 : 1) * kBoxes * box_bytes);
        for (int x = 0; x < (has_b ? 2 : 1); ++x) {
            const TileAt at = tile_at(g, qa + x);
#pragma unroll
            for (int c = 0; c < kBoxes; ++c)
                tma_load_4d(sbase + kQOff + x * kTile + c * kWBox, &tmQ, qbar, 64 * c, at.row, at.stripe, (int)bh);
        }
        // test hook: the first K/V tile is never loaded, so every wait on it
        // runs out (the kernel must then record the timeout and return)
        const bool skip_first = p.wc.inject == kInjectFwdSkipKV;
        int j = 0;
        for (; j < nt; ++j) {
            const int s = j % NS;
            if (j >= NS && !mbar_wait(smem_u32(&bars->kv_empty[s]), ((j / NS) + 1) & 1, p.wc)) break;
            if (skip_first && j == 0) continue;
            const TileAt at = tile_at(g, j < ns ? j : lo_a + j - ns);
            const uint32_t fb = smem_u32(&bars->kv_full[s]);
            const uint32_t kdst = sbase + kKVOff + s * kStage, vdst = kdst + kTile;
            mbar_arrive_expect_tx(fb, 2 * kBoxes * box_bytes);
#pragma unroll
            for (int c = 0; c < kBoxes; ++c) {
                tma_load_4d(kdst + c * kWBox, &tmK, fb, 64 * c, at.row, at.stripe, kvh);
                tma_load_4d(vdst + c * kWBox, &tmV, fb, 64 * c, at.row, at.stripe, kvh);
            }
        }
        // loads [0, j) and Q were issued: wait (bounded) for the last of each
        // stage, so that on an error path none lands after the CTA has exited
        mbar_wait(qbar, 0, p.wc);
        for (int t = j > NS ? j - NS : 0; t < j; ++t)
            if (!(skip_first && t == 0)) mbar_wait(smem_u32(&bars->kv_full[t % NS]), (t / NS) & 1, p.wc);
    } else if (warp == 1 && lane == 0) {
        // ---------------- MMA issuer: PV_A(j), S_A(next), PV_B(j), S_B(next)
        constexpr uint32_t idesc_qk = idesc_bf16_f32(WB, WB, false, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(WB, HD, false, true);
        int done[2] = {0, 0};  // tiles each group has finished
        bool ok = mbar_wait(smem_u32(&bars->q_full), 0, p.wc);
        tc_fence_after();
        auto issue_s = [&](int x, int t) -> bool {
            const int s = t % NS;
            if (!mbar_wait(smem_u32(&bars->kv_full[s]), (t / NS) & 1, p.wc)) return false;
            tc_fence_after();
            const uint32_t qaddr = sbase + kQOff + x * kTile;
            const uint32_t kaddr = sbase + kKVOff + s * kStage;
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t off = (kk >> 2) * kWBox + (kk & 3) * 32;
                mma_ss(tmem + 128 * x, sdesc_sw128(qaddr + off, 16, 1024), sdesc_sw128(kaddr + off, 16, 1024),
                       idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit(smem_u32(&bars->s_full[x]));
            return true;
        };
        auto issue_pv = [&](int x, int t) -> bool {
            if (!mbar_wait(smem_u32(&bars->p_ready[x]), done[x] & 1, p.wc)) return false;
            tc_fence_after();
            const uint32_t vaddr = sbase + kKVOff + (t % NS) * kStage + kTile;
#pragma unroll
            for (int kk = 0; kk < WB / 16; ++kk)
                mma_ts(tmem + 256 + 128 * x, tmem + 128 * x + kk * 8, sdesc_sw128(vaddr + kk * 2048, kWBox, 1024),
                       idesc_pv, (done[x] > 0 || kk > 0) ? 1u : 0u);
            mma_commit(smem_u32(&bars->o_done[x]));
            ++done[x];
            return true;
        };
        auto next_b = [&](int j) { return j + 1 == skip ? j + 2 : j + 1; };
        if (ok) ok = issue_s(0, 0);
        if (ok && has_b) ok = issue_s(1, next_b(-1));
        for (int j = 0; j < nt && ok; ++j) {
            if (j < n_a) {
                if (!issue_pv(0, j)) break;
                if (j + 1 < n_a && !issue_s(0, j + 1)) break;
            }
            const bool b = has_b && j != skip;
            if (b && !issue_pv(1, j)) break;
            // only stages the producer will refill get a release
            if (j + NS < nt) mma_commit(smem_u32(&bars->kv_empty[j % NS]));
            if (b && next_b(j) < nt && !issue_s(1, next_b(j))) break;
        }
        // every MMA issued above completes before TMEM is freed (error paths)
        mma_commit(smem_u32(&bars->drain));
        mbar_wait(smem_u32(&bars->drain), 0, p.wc);
    } else if (warp >= 2 && (warp < 6 || has_b)) {
        // ---------------- softmax + epilogue of one query tile
        const int x = (warp - 2) >> 2;       // group: query tile qa or qb
        const int qt = qa + x;
        const int quarter = warp & 3;
        const int ri = quarter * 32 + lane;  // query row of the tile
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + 128 * x + lane_off, tO = tmem + 256 + 128 * x + lane_off;
        const float cl2 = p.scale * 1.4426950408889634f;
        const int base = qt * g.P;                // first position of the tile
        const int pq = base + tile_pos(g, ri);    // position of this row (rows past the tile are not stored)
        float m_ref = -INFINITY, l = 0.f;
        int n = 0;  // tiles turned into P
        bool ok = true;
        const int j1 = x ? nt : n_a;
        for (int j = 0; j < j1; ++j) {
            if (x && j == skip) continue;
            const int kt = j < ns ? j : lo_a + j - ns;
            if (!mbar_wait(smem_u32(&bars->s_full[x]), n & 1, p.wc)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float sv[WB];
            {
                uint32_t r0[32], r1[32], r2[32], r3[32];
                tmem_ld32(tS, r0);
                tmem_ld32(tS + 32, r1);
                tmem_ld32(tS + 64, r2);
                tmem_ld32(tS + 96, r3);
                tmem_ld_wait(r0);
                tmem_ld_wait(r1);
                tmem_ld_wait(r2);
                tmem_ld_wait(r3);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    sv[c] = __uint_as_float(r0[c]);
                    sv[32 + c] = __uint_as_float(r1[c]);
                    sv[64 + c] = __uint_as_float(r2[c]);
                    sv[96 + c] = __uint_as_float(r3[c]);
                }
            }
            // kept columns: position <= pq and (>= pq - W + 1 or < sinks);
            // uniform test: every pair of the two tiles is kept
            const int kbase = kt * g.P;
            const bool full = g.P == WB && kt < qt &&
                              (kbase >= base + g.P - p.W || kbase + g.P <= p.sinks);
            if (!full) {
                const int hi = pq - kbase, lo = pq - p.W + 1 - kbase, sk = p.sinks - kbase;
#pragma unroll
                for (int c = 0; c < WB; c += 4) {
                    const int4 kp = *reinterpret_cast<const int4 *>(col_pos + c);
                    if (!(kp.x <= hi && (kp.x >= lo || kp.x < sk))) sv[c] = -INFINITY;
                    if (!(kp.y <= hi && (kp.y >= lo || kp.y < sk))) sv[c + 1] = -INFINITY;
                    if (!(kp.z <= hi && (kp.z >= lo || kp.z < sk))) sv[c + 2] = -INFINITY;
                    if (!(kp.w <= hi && (kp.w >= lo || kp.w < sk))) sv[c + 3] = -INFINITY;
                }
            }
            float mx8[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) mx8[t] = sv[t];
#pragma unroll
            for (int c = 8; c < WB; c += 16)
#pragma unroll
                for (int t = 0; t < 8; ++t) mx8[t] = fmax3(mx8[t], sv[c + t], sv[c + 8 + t]);
            const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                   fmaxf(mx8[6], mx8[7]));
            const float m_tile = mx * cl2;
            const bool move = n == 0 || m_tile > m_ref + kWRescale;
            const float m_new = move ? fmaxf(m_ref, m_tile) : m_ref;
            const float alpha = (n == 0 || !move) ? 1.f : ex2(m_ref - m_new);
            const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
            const uint64_t cl2x2 = f2(cl2, cl2), nm2 = f2(-m_use, -m_use);
            uint64_t acc4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float2 e = f2_split(fma2(f2(sv[64 * h + 2 * c], sv[64 * h + 2 * c + 1]), cl2x2, nm2));
                    const float p0 = ex2(e.x), p1 = ex2(e.y);
                    acc4[c & 3] = add2(acc4[c & 3], f2(p0, p1));
                    pk[c] = pack_bf16x2(p0, p1);
                }
                tmem_st32(tS + 32 * h, pk);
            }
            const float2 s01 = f2_split(add2(acc4[0], acc4[1])), s23 = f2_split(add2(acc4[2], acc4[3]));
            const float sum = (s01.x + s01.y) + (s23.x + s23.y);
            tmem_st_wait();
            l = l * alpha + sum;
            m_ref = m_new;
            if (n > 0) {
                // the group's previous PV must be complete before O is touched
                if (!mbar_wait(smem_u32(&bars->o_done[x]), (n - 1) & 1, p.wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < HD / 32; ++c) {
                        uint32_t rr[32];
                        tmem_ld32(tO + c * 32, rr);
                        tmem_ld_wait(rr);
#pragma unroll
                        for (int v = 0; v < 32; ++v) rr[v] = __float_as_uint(__uint_as_float(rr[v]) * alpha);
                        tmem_st32(tO + c * 32, rr);
                    }
                    tmem_st_wait();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->p_ready[x]));
            ++n;
        }
        // ---------------- epilogue
        if (ok) {
            ok = mbar_wait(smem_u32(&bars->o_done[x]), (n - 1) & 1, p.wc);
            tc_fence_after();
        }
        const bool valid = tile_has(g, qt, ri);
        const bool empty = !(l > 0.f) || !ok;
        const float inv_l = empty ? 0.f : 1.f / l;
        const float lse_row = empty ? -INFINITY : (m_ref + log2f(l)) * 0.6931471805599453f;
        const int64_t row = bh * (int64_t)g.S + (valid ? tile_row(g, qt, ri) : 0);
        if (valid) p.lse[row] = lse_row;
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
            uint32_t rr[32];
            tmem_ld32(tO + c * 32, rr);
            tmem_ld_wait(rr);
            if (!valid) continue;
            uint4 *dst = reinterpret_cast<uint4 *>(p.o + row * HD + c * 32);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                uint4 w;
                w.x = pack_bf16x2(__uint_as_float(rr[8 * v + 0]) * inv_l, __uint_as_float(rr[8 * v + 1]) * inv_l);
                w.y = pack_bf16x2(__uint_as_float(rr[8 * v + 2]) * inv_l, __uint_as_float(rr[8 * v + 3]) * inv_l);
                w.z = pack_bf16x2(__uint_as_float(rr[8 * v + 4]) * inv_l, __uint_as_float(rr[8 * v + 5]) * inv_l);
                w.w = pack_bf16x2(__uint_as_float(rr[8 * v + 6]) * inv_l, __uint_as_float(rr[8 * v + 7]) * inv_l);
                dst[v] = w;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD>
int launch_window_hd(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const WinParams &p,
                     int64_t nblocks, cudaStream_t stream) {
    static PerDeviceOnce once;
    const int attr = once.get([] {
        return cuda_status(cudaFuncSetAttribute(tc_window_fwd_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)WinCfg<HD>::kSmemBytes));
    });
    if (attr != STRIPED_OK) return attr;
    tc_window_fwd_kernel<HD><<<(unsigned)nblocks, kWThreads, WinCfg<HD>::kSmemBytes, stream>>>(mq, mk, mv, p);
    return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_tc_window_fwd(const void *q, const void *k, const void *v, void *o, float *lse, const WindowArgs &a,
                         cudaStream_t stream) {
    WinParams p{};
    if (!pos_geom(&p.g, a.S, a.N, a.layout)) return STRIPED_ERR_UNSUPPORTED;
    p.W = (int)(a.window < a.S ? a.window : a.S);
    p.sinks = (int)(a.sinks < a.S ? a.sinks : a.S);
    p.nst = (p.sinks + p.g.P - 1) / p.g.P;
    p.npair = (p.g.nt + 1) / 2;
    p.G = (int)(a.H / a.Hkv);
    p.scale = a.scale;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.wc = device_wait_ctl();
    const int64_t nblocks = (int64_t)p.npair * a.B * a.H;
    if (nblocks > 0x7fffffffll) return STRIPED_ERR_UNSUPPORTED;
    CUtensorMap mq, mk, mv;
    int st;
    if ((st = make_pos_map(&mq, q, a.D, p.g, a.B * a.H)) || (st = make_pos_map(&mk, k, a.D, p.g, a.B * a.Hkv)) ||
        (st = make_pos_map(&mv, v, a.D, p.g, a.B * a.Hkv)))
        return st;
    return a.D == 128 ? launch_window_hd<128>(mq, mk, mv, p, nblocks, stream)
                      : launch_window_hd<64>(mq, mk, mv, p, nblocks, stream);
}

}  // namespace striped
