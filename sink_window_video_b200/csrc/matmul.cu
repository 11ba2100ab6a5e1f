// matmul.cu -- products of NVFP4 matrices on the block-scaled FP4 tensor cores
// (tcgen05.mma kind::mxf4nvf4), with the epilogue fused, dense and grouped by
// expert:
//   Y[m][n] = R[m][n] + g * act(s_X s_W sum_k x[m][k] w[n][k] + b[n]),
// x and w the E2M1 codes times their E4M3 block scales (16 elements along k).
//
// The tensor core's A operand is the WEIGHT tile (128 output channels) and B
// the token tile (TN rows of X): a tensor-memory lane is then an output
// channel and a column a token, so one kernel serves one token and thousands
// (the token count only sets the instruction's N), a thread's bias is one
// register, and the 32 lanes of a warp store 32 neighbouring channels of one
// row of Y.
//
// One persistent CTA per SM over a static tile list; roles by warp:
//   warps 0-3  block scales, a stage each in turn: global -> registers ->
//              shared memory in the tensor core's scale layout (below)
//   warp 4     TMA loads of both code tiles (lane 0)
//   warp 5     tcgen05.cp of the scales into tensor memory and the MMAs (lane 0)
//   warps 8-15 epilogue: tensor memory -> registers -> Y
// A stage holds 256 elements along k: 128 bytes of codes a row (one 128-byte
// swizzle row) and 16 scale bytes a row.  Two accumulators in tensor memory
// let the epilogue of one tile run under the next tile's MMAs.
// Scale layout of one K = 64 step and 128 rows: 512 bytes, row r's four block
// scales (bytes) at (r % 32) * 16 + (r / 32) * 4, which tcgen05.cp
// (32x128b.warpx4) places in 4 columns of every lane quarter.
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace nvfp4kv {
using namespace tc;
namespace {

constexpr int kTileN = 128;                 // output channels of a tile (the MMA's M)
constexpr int kStageK = 256;                // elements along k of one stage
constexpr int kThreadsMM = 512;
constexpr int kScaleWarps = 4, kTmaWarp = 4, kMmaWarp = 5, kEpiWarp0 = 8;   // 6, 7: idle
// Registers of a thread: 128 at launch (65536 / 512), 80 for the first two
// warpgroups and 176 for the epilogue's (256 * 80 + 256 * 176 = 65536).
constexpr int kFewRegs = 80, kManyRegs = 176;
constexpr int kColsMM = 512;                // tensor-memory columns
constexpr uint32_t kColSFAm = 448, kColSFBm = 464;   // 16 and 32 columns
constexpr int kATile = kTileN * 128;        // bytes of codes of a weight tile's stage
constexpr int kSfaBytes = 4 * 512;
constexpr int kMaxStages = 12;

template <int TN>
struct Shape {
    static constexpr int kBTile = TN * 128;
    static constexpr int kSfbBytes = 4 * 512 * ((TN + 127) / 128);
    static constexpr int kStage = kATile + kBTile + kSfaBytes + kSfbBytes;
    static constexpr int kStages = (200 * 1024) / kStage < kMaxStages ? (200 * 1024) / kStage
                                                                      : kMaxStages;
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
    // a scale warp waits for the stage's last use by its parity alone, which is
    // unambiguous only while no warp is more than kStages steps ahead
    static_assert(kScaleWarps <= kStages, "one phase of a stage at a time");
    static_assert(kStage % 1024 == 0, "stages keep the swizzle alignment");
    static_assert(2 * TN <= (int)kColSFAm, "two accumulators beside the scales");
};

struct MMShared {
    uint64_t tma_full[kMaxStages];
    uint64_t sf_full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_free[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int bad_offsets;
};

__device__ __forceinline__ bool wait_or_abort_m(uint32_t mbar, uint32_t parity, volatile int* abort,
                                                Control* ctl, unsigned site, unsigned step) {
    if (mbar_try_wait(mbar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (mbar_try_wait(mbar, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            record_timeout(ctl, site, step, parity);
            return false;
        }
    }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar)
        : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred P;\nelect.sync _|P, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, P;\n}" : "=r"(p));
    return p != 0;
}

template <int R>
__device__ __forceinline__ void reg_dealloc() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void reg_alloc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mbar), "r"(bytes)
                 : "memory");
}

// 512 bytes (32 rows of 16) of shared memory into 4 columns of all four lane
// quarters.
__device__ __forceinline__ void tmem_cp_scales(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc));
}

// Four consecutive block scales of one row from byte kb of it (zeros from
// byte kbytes on).  kbytes is even (K a multiple of 32).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int kb, int kbytes) {
    const int left = kbytes - kb;
    if (left <= 0) return 0u;
    if ((kbytes & 3) == 0) return __ldg(reinterpret_cast<const uint32_t*>(row + kb));
    const uint32_t lo = __ldg(reinterpret_cast<const uint16_t*>(row + kb));
    const uint32_t hi = left > 2 ? __ldg(reinterpret_cast<const uint16_t*>(row + kb + 2)) : 0u;
    return lo | (hi << 16);
}

// The 16 block scales of one stage of one row.
__device__ __forceinline__ uint4 scale_row(const uint8_t* row, int kb, int kbytes) {
    if ((kbytes & 15) == 0) return __ldg(reinterpret_cast<const uint4*>(row + kb));
    return make_uint4(scale_word(row, kb, kbytes), scale_word(row, kb + 4, kbytes),
                      scale_word(row, kb + 8, kbytes), scale_word(row, kb + 12, kbytes));
}

// z * sigmoid(v) for two values, v = z (SiLU) or 2 sqrt(2/pi) (z + 0.044715 z^3)
// (GELU, tanh form: (1 + tanh(v/2)) / 2 = sigmoid(v)).  The two quotients share
// one reciprocal, 1/a = b / (a b), since the special-function unit is what a
// tile's activation waits for (1.5 instead of 2 operations a value); -v log2 e
// is held to 60, so that a b stays finite: sigmoid below 2^-60 is lost to z's
// last place many times over.
template <int kAct>
__device__ __forceinline__ float2 act_pair(float2 z) {
    if (kAct == NVFP4KV_ACT_NONE) return z;
    float2 x;
    if (kAct == NVFP4KV_ACT_SILU) {
        x = __fmul2_rn(z, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    } else {
        constexpr float c1 = -1.4426950408889634f * 1.5957691216057308f;
        constexpr float c3 = c1 * 0.044715f;
        const float2 z2 = __fmul2_rn(z, z);
        x = __fmul2_rn(z, __ffma2_rn(z2, make_float2(c3, c3), make_float2(c1, c1)));
    }
    const float2 e = make_float2(ex2f(fminf(x.x, 60.0f)), ex2f(fminf(x.y, 60.0f)));
    const float2 d = __fadd2_rn(e, make_float2(1.0f, 1.0f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d.x * d.y));
    return __fmul2_rn(z, __fmul2_rn(make_float2(d.y, d.x), make_float2(r, r)));
}

template <bool kF32>
struct OutType {
    using T = float;
};
template <>
struct OutType<false> {
    using T = __nv_bfloat16;
};
__device__ __forceinline__ float load_out(const float* p) { return *p; }
__device__ __forceinline__ float load_out(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The next row's address.  The empty asm keeps the compiler from forming every
// multiple of the row stride ahead of the loops (two registers each).
template <class T>
__device__ __forceinline__ void next_row(T*& p, long long ld) {
    p += ld;
    asm("" : "+l"(p));
}

constexpr int kChunk = 16;      // tokens an epilogue warp takes at a time

// Tokens m .. m + C - 1 of one channel, accumulators in tensor memory at taddr.
// kTest: tokens from m_end on and channels from N on are left out, and the gate
// is looked up for each token; otherwise the C tokens are whole and share the
// gate g.  The residual's (and gates') loads are all in flight while the
// accumulators are read.
template <int C, bool kF32, int kAct, bool kGrouped, bool kTest>
__device__ __forceinline__ void epilogue_tokens(const MatmulArgs& a, uint32_t taddr, int m, int m_end,
                                                int n, float alpha, float b, float g) {
    using T = typename OutType<kF32>::T;
    const int count = kTest ? (n < a.N ? m_end - m : 0) : C;
    uint32_t v[C];
    if (C == 32) tmem_ld32(taddr, v);
    else tmem_ld16(taddr, v);
    T* y = static_cast<T*>(a.Y) + (size_t)m * a.ldy + n;
    T res[C];
    if (a.residual) {
        const T* r = static_cast<const T*>(a.residual) + (size_t)m * a.ldr + n;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if (!kTest || j < count) res[j] = *r;
            next_row(r, a.ldr);
        }
    }
    constexpr bool kGates = kTest && !kGrouped;
    float gates[kGates ? C : 1];
    if (kGates && a.gate) {
        int q = m / a.rows_per_gate, rem = m - q * a.rows_per_gate;
        const float* gp = a.gate + (size_t)q * a.N + n;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if (j < count) gates[j] = __ldg(gp);
            if (++rem == a.rows_per_gate) {
                rem = 0;
                next_row(gp, a.N);
            }
        }
    }
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < C; j += 2) {
        float2 z = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                              make_float2(alpha, alpha), make_float2(b, b));
        z = act_pair<kAct>(z);
        float2 gg = make_float2(g, g);
        if (kGates && a.gate) gg = make_float2(gates[j], gates[j + 1]);
        if (a.residual)
            z = __ffma2_rn(z, gg, make_float2(load_out(&res[j]), load_out(&res[j + 1])));
        else
            z = __fmul2_rn(z, gg);
        if (!kTest || j < count) store_out(y, z.x);
        next_row(y, a.ldy);
        if (!kTest || j + 1 < count) store_out(y, z.y);
        next_row(y, a.ldy);
    }
}

template <bool kF32, int kAct, bool kGrouped>
__device__ __forceinline__ void epilogue_chunk(const MatmulArgs& a, uint32_t taddr, int m, int m_end,
                                               int n, float alpha, float b, float g, bool whole) {
    if (whole) {
        epilogue_tokens<kChunk, kF32, kAct, kGrouped, false>(a, taddr, m, m_end, n, alpha, b, g);
    } else {
#pragma unroll 1
        for (int c = 0; c < kChunk && m + c < m_end; c += 16) {
            epilogue_tokens<16, kF32, kAct, kGrouped, true>(a, taddr + c, m + c, m_end, n, alpha, b,
                                                            g);
            __syncwarp();
        }
    }
}

struct TileAt {
    int e, n0, m0, m_end;
};

template <int TN, bool kGrouped>
struct Tiles {
    const MatmulArgs& a;
    const int* s_off;
    const int* s_tile;
    int n_tiles, e;
    __device__ Tiles(const MatmulArgs& args, const int* off, const int* tile)
        : a(args), s_off(off), s_tile(tile), e(0) {
        n_tiles = (a.N + kTileN - 1) / kTileN;
    }
    __device__ int total() const {
        return kGrouped ? s_tile[a.E] : ((a.M + TN - 1) / TN) * n_tiles;
    }
    // t grows from call to call
    __device__ TileAt at(int t) {
        TileAt r;
        int row0 = 0, m_end = a.M;
        if (kGrouped) {
            while (s_tile[e + 1] <= t) ++e;
            t -= s_tile[e];
            row0 = s_off[e];
            m_end = s_off[e + 1];
        }
        const int mt = t / n_tiles;
        r.e = e;
        r.n0 = (t - mt * n_tiles) * kTileN;
        r.m0 = row0 + mt * TN;
        r.m_end = min(m_end, r.m0 + TN);
        return r;
    }
};

template <int TN, bool kGrouped, bool kF32>
__global__ void __launch_bounds__(kThreadsMM, 1)
matmul_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
              const MatmulArgs a) {
    using S = Shape<TN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ MMShared sh;
    __shared__ int s_off[kGrouped ? kMaxExperts + 1 : 1];
    __shared__ int s_tile[kGrouped ? kMaxExperts + 1 : 1];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &sh.abort;
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);

    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem_base)),
                     "r"(kColsMM));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        sh.abort = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_u32(&sh.tma_full[s]), 1);
            mbar_init(smem_u32(&sh.sf_full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.acc_full[i]), 1);
            mbar_init(smem_u32(&sh.acc_free[i]), 8);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (kGrouped && warp == 0) {
        // tile count prefix over the experts; offsets that decrease or leave
        // [0, M] are reported and nothing is computed
        const int nt = (a.N + kTileN - 1) / kTileN;
        int carry = 0;
        bool bad = false;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            int cnt = 0;
            if (e < a.E) {
                const int o0 = a.offsets[e], o1 = a.offsets[e + 1];
                bad |= o0 < 0 || o1 < o0 || o1 > a.M;
                s_off[e] = o0;
                if (e == a.E - 1) s_off[a.E] = o1;
                cnt = ((o1 - o0 + TN - 1) / TN) * nt;
            }
            int inc = cnt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                if (lane >= d) inc += v;
            }
            if (e < a.E) s_tile[e + 1] = carry + inc;
            carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
        bad = __any_sync(0xFFFFFFFFu, bad);
        if (lane == 0) {
            s_tile[0] = 0;
            if (bad) {
                s_tile[a.E] = 0;
                if (blockIdx.x == 0) atomicOr(&a.ctl->status, kStatusOffsets);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    Tiles<TN, kGrouped> tiles(a, s_off, s_tile);
    const int total = tiles.total();
    const int steps = (a.K + kStageK - 1) / kStageK;
    const int kbytes = a.K / 16;

    if (warp < kEpiWarp0) reg_dealloc<kFewRegs>();
    else reg_alloc<kManyRegs>();
    if (warp < kTmaWarp) {
        // ------------------------------------------------------------ block scales
        // warp w takes every kScaleWarps-th stage: lane l has rows l, 32 + l, ..
        // of the weight and the token tile, 16 bytes each, loaded while the
        // warps before it hold the turn; four rows' words of one K = 64 step
        // are one 16-byte line of the layout
        constexpr int kXRows = TN / 32;
        constexpr int kSfbGroups = (TN + 127) / 128;
        const bool withhold = blockIdx.x == 0 && warp == 0 && (a.ctl->test_flags & 1u) != 0u;
        uint4 wv[4], xv[kXRows];
        auto load = [&](const TileAt& at, int s) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = at.n0 + 32 * i + lane;
                wv[i] = make_uint4(0u, 0u, 0u, 0u);
                if (n < a.N)
                    wv[i] = scale_row(a.w_scales + ((size_t)at.e * a.w_scale_rows +
                                                    (n >> a.w_shift)) * kbytes,
                                      s * 16, kbytes);
            }
#pragma unroll
            for (int i = 0; i < kXRows; ++i) {
                const int m = at.m0 + 32 * i + lane;
                xv[i] = make_uint4(0u, 0u, 0u, 0u);
                if (m < at.m_end)
                    xv[i] = scale_row(a.x_scales + (size_t)(m >> a.x_shift) * kbytes, s * 16, kbytes);
            }
        };
        auto put4 = [&](uint8_t* dst, int stride, const uint4& r0, const uint4& r1, const uint4& r2,
                        const uint4& r3) {
            uint4* d = reinterpret_cast<uint4*>(dst + lane * 16);
            const int q = stride / 16;
            d[0] = make_uint4(r0.x, r1.x, r2.x, r3.x);
            d[q] = make_uint4(r0.y, r1.y, r2.y, r3.y);
            d[2 * q] = make_uint4(r0.z, r1.z, r2.z, r3.z);
            d[3 * q] = make_uint4(r0.w, r1.w, r2.w, r3.w);
        };
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        // (t, s): tile and stage of step it
        int t = blockIdx.x, s = warp;
        auto settle = [&] {
            while (s >= steps && t < total) {
                s -= steps;
                t += gridDim.x;
            }
        };
        settle();
        int t_at = -1;
        TileAt at;
        auto fetch = [&] {
            if (t >= total) return;
            if (t != t_at) at = tiles.at(t);
            t_at = t;
            load(at, s);
        };
        fetch();
        for (int it = warp; t < total; it += kScaleWarps) {
            const int st = it % S::kStages;
            if (it >= S::kStages) {
                bool ok = wait_or_abort_m(smem_u32(&sh.empty[st]),
                                          (uint32_t)((it / S::kStages - 1) & 1), abort, a.ctl, 60u, it);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
            }
            uint8_t* sf = base + (size_t)st * S::kStage + kATile + S::kBTile;
            put4(sf, 512, wv[0], wv[1], wv[2], wv[3]);
#pragma unroll
            for (int i = 0; i < kSfbGroups; ++i)
                put4(sf + kSfaBytes + 512 * i, 512 * kSfbGroups, xv[4 * i],
                     4 * i + 1 < kXRows ? xv[(4 * i + 1) % kXRows] : none,
                     4 * i + 2 < kXRows ? xv[(4 * i + 2) % kXRows] : none,
                     4 * i + 3 < kXRows ? xv[(4 * i + 3) % kXRows] : none);
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && !(withhold && it == 0)) mbar_arrive(smem_u32(&sh.sf_full[st]));
            s += kScaleWarps;
            settle();
            fetch();
        }
    } else if (warp >= kEpiWarp0) {
        // ------------------------------------------------------------ epilogue
        // warp = lane quarter (warp % 4) of every second chunk of the tokens
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        int i = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++i) {
            const TileAt at = tiles.at(t);
            const int buf = i & 1;
            const int n = at.n0 + (warp & 3) * 32 + lane;
            const bool nv = n < a.N;
            const bool warp_nv = at.n0 + (warp & 3) * 32 + 31 < a.N;
            const size_t en = (size_t)at.e * a.N + n;
            const float alpha = __ldg(a.x_scale) * __ldg(a.w_scale + at.e);
            const float b = (a.bias && nv) ? __ldg(a.bias + en) : 0.0f;
            float g = (a.gate && kGrouped && nv) ? __ldg(a.gate + en) : 1.0f;
            bool got = wait_or_abort_m(smem_u32(&sh.acc_full[buf]), (uint32_t)((i >> 1) & 1), abort,
                                       a.ctl, 61u, i);
            if (!__all_sync(0xFFFFFFFFu, got)) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = (warp >> 2) % 2 * kChunk; c < TN && at.m0 + c < at.m_end; c += 2 * kChunk) {
                const int m = at.m0 + c;
                bool whole = warp_nv && m + kChunk <= at.m_end;
                if (!kGrouped && a.gate && whole) {
                    const int row = m / a.rows_per_gate;
                    whole = (m + kChunk - 1) / a.rows_per_gate == row;
                    g = __ldg(a.gate + (size_t)row * a.N + n);
                }
                const uint32_t ta = tmem + lane_base + (uint32_t)(buf * TN + c);
                if (a.act == NVFP4KV_ACT_GELU_TANH)
                    epilogue_chunk<kF32, NVFP4KV_ACT_GELU_TANH, kGrouped>(a, ta, m, at.m_end, n, alpha, b, g, whole);
                else if (a.act == NVFP4KV_ACT_SILU)
                    epilogue_chunk<kF32, NVFP4KV_ACT_SILU, kGrouped>(a, ta, m, at.m_end, n, alpha, b, g,
                                                                          whole);
                else
                    epilogue_chunk<kF32, NVFP4KV_ACT_NONE, kGrouped>(a, ta, m, at.m_end, n, alpha, b, g,
                                                                          whole);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.acc_free[buf]));
        }
    } else if (warp == kTmaWarp) {
        // ------------------------------------------------------------ code tiles
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const TileAt at = tiles.at(t);
                for (int s = 0; s < steps; ++s, ++it) {
                    const int st = it % S::kStages;
                    if (it >= S::kStages) {
                        ok = wait_or_abort_m(smem_u32(&sh.empty[st]),
                                             (uint32_t)((it / S::kStages - 1) & 1), abort, a.ctl, 62u,
                                             it);
                        if (!ok) break;
                    }
                    const uint32_t dst = smem_u32(base + (size_t)st * S::kStage);
                    const uint32_t bar = smem_u32(&sh.tma_full[st]);
                    mbar_expect_tx(bar, (uint32_t)(kATile + S::kBTile));
                    tma_load_3d(dst, &map_w, s * 128, at.n0, at.e, bar);
                    tma_load_3d(dst + kATile, &map_x, s * 128, at.m0, 0, bar);
                }
            }
            if (!ok) {
                // the loads in flight land before the CTA leaves
                const int first = it > S::kStages ? it - S::kStages : 0;
                for (int i = first; i < it; ++i)
                    mbar_wait(smem_u32(&sh.tma_full[i % S::kStages]),
                              (uint32_t)((i / S::kStages) & 1));
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issue
        // the whole warp walks the steps; one elected lane issues
        constexpr uint32_t idesc = umma_idesc_fp4(TN);
        constexpr int kSfbGroups = (TN + 127) / 128;
        int it = 0, i = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++i) {
            const int buf = i & 1;
            if (i >= 2) {
                ok = wait_or_abort_m(smem_u32(&sh.acc_free[buf]), (uint32_t)((i / 2 - 1) & 1),
                                     abort, a.ctl, 63u, i);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
            }
            const uint32_t d = tmem + (uint32_t)(buf * TN);
            for (int s = 0; s < steps; ++s, ++it) {
                const int st = it % S::kStages;
                const uint32_t par = (uint32_t)((it / S::kStages) & 1);
                ok = wait_or_abort_m(smem_u32(&sh.sf_full[st]), par, abort, a.ctl, 64u, it) &&
                     wait_or_abort_m(smem_u32(&sh.tma_full[st]), par, abort, a.ctl, 65u, it);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sa = smem_u32(base + (size_t)st * S::kStage);
                const uint32_t sf = sa + kATile + S::kBTile;
                const uint64_t da = umma_desc(sa, 16, 1024);
                const uint64_t db = umma_desc(sa + kATile, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        tmem_cp_scales(tmem + kColSFAm + 4u * j,
                                       umma_desc_noswizzle(sf + 512 * j, 16, 128));
#pragma unroll
                        for (int q = 0; q < kSfbGroups; ++q)
                            tmem_cp_scales(tmem + kColSFBm + 8u * j + 4u * q,
                                           umma_desc_noswizzle(
                                               sf + kSfaBytes + 512 * (kSfbGroups * j + q), 16, 128));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_fp4(d, da + 2u * j, db + 2u * j, idesc, (s | j) ? 1u : 0u,
                                tmem + kColSFAm + 4u * j, tmem + kColSFBm + 8u * j);
                    mma_commit(smem_u32(&sh.empty[st]));
                    if (s == steps - 1) mma_commit(smem_u32(&sh.acc_full[buf]));
                }
                __syncwarp();
            }
        }
        if (elect_one()) mma_commit(smem_u32(&sh.drain));
        __syncwarp();
        mbar_wait(smem_u32(&sh.drain), 0u);
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kColsMM));
    }
}

// ------------------------------------------------------------------ host

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// Codes [depth][rows][K / 2] as bytes, tiles of `box` rows of 128 bytes with
// the 128-byte swizzle; what lies outside reads as zero codes.
bool make_map(CUtensorMap* map, const void* codes, int K, int rows, int depth, int box) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)K / 2, (cuuint64_t)rows, (cuuint64_t)depth};
    const cuuint64_t strides[2] = {(cuuint64_t)K / 2, (cuuint64_t)K / 2 * rows};
    const cuuint32_t boxes[3] = {128, (cuuint32_t)box, 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, boxes,
              ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// Multiprocessors of a device, asked for once (0: no answer).
int sm_count_of(int dev) {
    static std::atomic<int> known[kMaxDevices];
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Allow the kernel its shared memory, once on each device.
template <int TN, bool kGrouped, bool kF32>
bool configure(int dev) {
    static std::atomic<bool> done[kMaxDevices];
    if (done[dev].load(std::memory_order_relaxed)) return true;
    if (cudaFuncSetAttribute(matmul_kernel<TN, kGrouped, kF32>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Shape<TN>::kSmem) != cudaSuccess)
        return false;
    done[dev].store(true, std::memory_order_relaxed);
    return true;
}

template <int TN, bool kGrouped, bool kF32>
nvfp4kv_status launch_tn(const MatmulArgs& a, const void* w_codes, const void* x_codes,
                         cudaStream_t stream) {
    CUtensorMap map_w, map_x;
    if (!make_map(&map_w, w_codes, a.K, a.N, kGrouped ? a.E : 1, kTileN) ||
        !make_map(&map_x, x_codes, a.K, a.M, 1, TN))
        return NVFP4KV_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices ||
        !configure<TN, kGrouped, kF32>(dev))
        return NVFP4KV_ERR_CUDA;
    const long long n_tiles = (a.N + kTileN - 1) / kTileN;
    // grouped: at most one more token tile per expert than the rows fill
    const long long most = n_tiles * ((a.M + TN - 1) / TN + (kGrouped ? a.E : 0));
    const int sms = sm_count_of(dev);
    const int grid = (int)(most < sms ? most : sms);
    if (grid <= 0) return NVFP4KV_ERR_CUDA;
    matmul_kernel<TN, kGrouped, kF32><<<grid, kThreadsMM, Shape<TN>::kSmem, stream>>>(map_w, map_x, a);
    return cudaGetLastError() == cudaSuccess ? NVFP4KV_OK : NVFP4KV_ERR_CUDA;
}

template <bool kGrouped, bool kF32>
nvfp4kv_status launch_any(const MatmulArgs& a, const void* w_codes, const void* x_codes,
                          cudaStream_t stream) {
    const int per = kGrouped ? (a.M + a.E - 1) / a.E : a.M;
    if (per <= 32) return launch_tn<32, kGrouped, kF32>(a, w_codes, x_codes, stream);
    if (per <= 128) return launch_tn<128, kGrouped, kF32>(a, w_codes, x_codes, stream);
    return launch_tn<192, kGrouped, kF32>(a, w_codes, x_codes, stream);
}

}  // namespace

nvfp4kv_status launch_matmul(const MatmulArgs& a, const void* w_codes, const void* x_codes,
                             cudaStream_t stream) {
    if (a.offsets)
        return a.y_f32 ? launch_any<true, true>(a, w_codes, x_codes, stream)
                       : launch_any<true, false>(a, w_codes, x_codes, stream);
    return a.y_f32 ? launch_any<false, true>(a, w_codes, x_codes, stream)
                   : launch_any<false, false>(a, w_codes, x_codes, stream);
}

}  // namespace nvfp4kv
