// matmul.cu -- products of NVFP4 matrices on the block-scaled FP4 tensor cores
// (tcgen05.mma kind::mxf4nvf4), with the epilogue fused, dense and grouped by
// expert:
//   Y[m][n] = R[m][n] + g * act(s_X s_W sum_k x[m][k] w[n][k] + b[n]),
// x and w the E2M1 codes times their E4M3 block scales (16 elements along k).
// The block products are exact in the tensor core and summed there in fp32 (5e-8
// off 64 bits relative to the result's norm at K = 8192); the epilogue is fp32.
//
// The tensor core's A operand is the WEIGHT tile (128 output channels a CTA) and
// B the token tile (up to TN rows of X): a tensor-memory lane is then an output
// channel and a column a token, so that one kernel serves one token and
// thousands: the tile's tokens, rounded up to 16, are the instruction's N.
//
// One persistent CTA per SM, or a pair of CTAs on two SMs for wide tiles
// (cta_group::2: 256 channels x TN tokens, each CTA staging its own channels and
// half of the tokens), over a static tile list; roles by warp:
//   warps 0-3  block scales: global -> registers (a turn ahead) -> shared
//              memory in the tensor core's scale layout (below)
//   warp 4     TMA loads of both code tiles (one elected lane)
//   warp 5     tcgen05.cp of the scales into tensor memory and the MMAs (one
//              elected lane; of a pair, the leader's: the other's hands its CTA's
//              scales over)
//   warp 6     the residual of the next tile into L2
//   warps 8-15 epilogue: tensor memory -> registers -> Y
// A stage holds 256 elements along k: 128 bytes of codes a row (one 128-byte
// swizzle row).  The block scales (16 bytes a row and stage) travel apart, 4
// stages at a turn, so that a row's 64 bytes are read together and the scale
// warps hand over once for 4 stages.  Two accumulators in tensor memory let the
// epilogue of one tile run under the next tile's MMAs.
// Scale layout of one K = 64 step and 128 rows: 512 bytes, row r's four block
// scales (bytes) at (r % 32) * 16 + (r / 32) * 4, which tcgen05.cp
// (32x128b.warpx4) places in 4 columns of every lane quarter.
//
// What bounds it.  [7040, 2048] x [8192, 2048] with GELU to bf16 takes 69 to 71 us
// (3.3 to 3.4 PFLOP/s, the bf16 tensor peak is 1.63), without its epilogue 47 us:
// epilogue and main loop share the SM's shared-memory pipe and issue slots.  A pair
// halves the shared-memory writes and reads of the token tile, which bound the single
// CTA ([7040, 8192] x [2048, 8192]: 70 us with 128 tokens on one CTA, 66 with a
// pair's 192).  Kept busy for seconds the first call takes 87 us: the clock falls to
// the power limit.  Small calls are latency: one row takes 5.0 to 5.2 us.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace nvfp4kv {
using namespace tc;
namespace {

constexpr int kTileN = 128;                 // output channels of a tile (the MMA's M)
constexpr int kStageK = 256;                // elements along k of one stage
constexpr int kThreadsMM = 512;
constexpr int kScaleWarps = 4, kTmaWarp = 4, kMmaWarp = 5, kEpiWarp0 = 8, kEpiWarps = 8;
constexpr int kPrefetchWarp = 6;            // (7: idle)
// Registers of a thread: 128 at launch (65536 / 512); 112 for the first two
// warpgroups (the scale warps hold a turn's 60 words) and 144 for the epilogue's
// two: 256 * 112 + 256 * 144 = 65536.
constexpr int kFewRegs = 112, kManyRegs = 144;
constexpr int kColsMM = 512;                // tensor-memory columns
constexpr int kATile = kTileN * 128;        // bytes of codes of a weight tile's stage
// Scales travel in turns of 4 steps; a K = 64 block of a 128-row group takes 512
// bytes, 16 more apart so that a warp's 16-byte lines fall in different banks.
constexpr int kTurn = 4;
constexpr int kSfBlock = 512 + 16;
constexpr int kSfGroup = 4 * kTurn * kSfBlock;
constexpr int kChunk = 16;                  // tokens an epilogue warp takes at a time
constexpr int kEpiBytes = 1024;             // its staging: 16 bf16 or 8 fp32 rows of 32
constexpr int kMaxStages = 12;
// After a wait that gave up, a CTA stays this long (10 ms) for its loads to land.
constexpr unsigned long long kLandNs = 10ull * 1000 * 1000;
constexpr size_t kStageRoom = 216 * 1024;    // of 227 KB; the rest: offsets, barriers, alignment

// Instruction descriptor of the block-scaled MMA (kind::mxf4nvf4, E2M1
// operands, E4M3 scales, fp32 D) for m x n.
__host__ __device__ constexpr uint32_t umma_idesc_scaled(uint32_t m, uint32_t n) {
    return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

template <int V>
struct IntC {
    static constexpr int value = V;
};

// Position in a ring of N slots and the parity of its current pass.
template <int N>
struct Ring {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            phase ^= 1u;
        }
    }
};

// TN tokens a tile; G CTAs (one, or a pair) share its MMAs: each has its own
// 128 output channels, and stages TN / G of the token rows.
template <int TN, int G>
struct Shape {
    static constexpr int kBTile = TN / G * 128;
    static constexpr int kStage = kATile + kBTile;
    static constexpr int kGroups = 1 + (TN + 127) / 128;     // 128-row groups of scales
    static constexpr int kSfStage = kGroups * kSfGroup;
    static constexpr int kFit = (int)((kStageRoom - 2 * kSfStage - kEpiWarps * kEpiBytes) / kStage);
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    static constexpr size_t kSmem = (size_t)kStages * kStage + 2 * kSfStage + kEpiWarps * kEpiBytes +
                                    1024;
    static_assert(kStage % 1024 == 0, "stages keep the swizzle alignment");
    static constexpr uint32_t kColSFA = 2 * TN, kColSFB = 2 * TN + 16;   // 16 and up to 32 columns
    static_assert(2 * TN + 16 + 8 * 4 <= kColsMM, "two accumulators beside the scales");
    static constexpr int kBox = TN / G % 32 == 0 ? 32 : 56;   // token rows of one TMA load
    static_assert(TN / G % kBox == 0, "whole loads of token rows");
};

struct MMShared {
    uint64_t tma_full[kMaxStages];
    uint64_t sf_full[2];
    uint64_t sf_own[2];      // of a pair's second CTA: its scales, before the leader's sf_full
    uint64_t sf_empty[2];
    uint64_t empty[kMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_free[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

// The address of rank 0's copy of a shared-memory object, in the cluster window.
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
                 : "memory");
}
// Arrive on the leader's barrier (for one CTA, its own) to free an accumulator.  No
// memory changes hands, so nothing has to be released to the other CTA: the sums
// are in registers (tcgen05.wait::ld) before the arrival, and what may overwrite
// them is issued after it was seen.
template <int G>
__device__ __forceinline__ void arrive_leader(uint32_t mbar) {
    if (G == 1) mbar_arrive(mbar);
    else mbar_arrive_cluster(leader_addr(mbar));
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// mbar_try_wait that the hardware may suspend for up to 20 us: a warp that waits
// then takes no issue slots from the epilogue.  kCluster: acquires what another CTA
// released (the MMA lane the second CTA's scales; what TMA and the tensor core bring
// or free comes with their own arrivals).
template <bool kCluster>
__device__ __forceinline__ bool try_wait_long(uint32_t mbar, uint32_t parity) {
    uint32_t ok;
    if (kCluster)
        asm volatile(
            "{\n.reg .pred P1;\n"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P1, [%1], %2, %3;\n"
            "selp.u32 %0, 1, 0, P1;\n}"
            : "=r"(ok)
            : "r"(mbar), "r"(parity), "r"(20000)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred P1;\nmbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2, %3;\n"
            "selp.u32 %0, 1, 0, P1;\n}"
            : "=r"(ok)
            : "r"(mbar), "r"(parity), "r"(20000)
            : "memory");
    return ok != 0;
}

// Wait for the mbarrier phase `parity`, for at most kWaitLimitNs or until another
// role of the CTA gave up.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_or_abort_m(uint32_t mbar, uint32_t parity, volatile int* abort,
                                                Control* ctl, unsigned site, unsigned step) {
    if (try_wait_long<kCluster>(mbar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    while (true) {
        if (try_wait_long<kCluster>(mbar, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            record_timeout(ctl, site, step, parity);
            return false;
        }
    }
}

template <int G>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t mbar) {
    if (G == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar)
            : "memory");
    else      // into this CTA, counted by the leader's barrier
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar)
            : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred P;\nelect.sync _|P, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, P;\n}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mbar), "r"(bytes)
                 : "memory");
}

// 512 bytes (32 rows of 16) of shared memory into 4 columns of all four lane
// quarters; for a pair each CTA's own shared memory into its own tensor memory.
template <int G>
__device__ __forceinline__ void tmem_cp_scales(uint32_t tmem, uint64_t desc) {
    if (G == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc));
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc));
}

// D (+)= (W scale_W) (X scale_X)^T; for a pair, D's 256 rows and the token rows
// lie half in each CTA.
template <int G>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc,
                                           uint32_t accumulate, uint32_t sfa, uint32_t sfb) {
    if (G == 1)
        mma_fp4(d, da, db, idesc, accumulate, sfa, sfb);
    else
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], "
            "p;\n}" ::"r"(d),
            "l"(da), "l"(db), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb));
}

// Arrive, when the MMAs and copies issued so far are done, on this barrier: of
// the issuing CTA, or of every CTA of the tile.
template <int G>
__device__ __forceinline__ void commit_own(uint32_t mbar) {
    if (G == 1)
        mma_commit(mbar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(mbar)
            : "memory");
}
template <int G>
__device__ __forceinline__ void commit_all(uint32_t mbar) {
    if (G == 1)
        mma_commit(mbar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
            "[%0], %1;" ::"r"(mbar),
            "h"((uint16_t)3)
            : "memory");
}

__device__ __forceinline__ void put_words(uint32_t* w, const uint4& v) {
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
}

// 16 bytes at p, or zeros.  One predicated load: as a branch around a load, the
// join of its two sides waits for the data, and a run of such loads goes one by
// one instead of together.
__device__ __forceinline__ uint4 load16_if(const uint8_t* p, bool yes) {
    uint4 v;
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %5, 0;\n"
        "mov.u32 %0, 0;\nmov.u32 %1, 0;\nmov.u32 %2, 0;\nmov.u32 %3, 0;\n"
        "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((int)yes));
    return v;
}

__device__ __forceinline__ uint32_t load4_if(const uint8_t* p, bool yes) {
    uint32_t v;
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\nmov.u32 %0, 0;\n@p ld.global.nc.u32 %0, [%1];\n}"
        : "=&r"(v)
        : "l"(p), "r"((int)yes));
    return v;
}

__device__ __forceinline__ uint32_t load2_if(const uint8_t* p, bool yes) {
    uint32_t v;
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\nmov.u32 %0, 0;\n@p ld.global.nc.u16 %0, [%1];\n}"
        : "=&r"(v)
        : "l"(p), "r"((int)yes));
    return v;
}

// The same for a residual, which may be Y itself (an ordinary load), and for a
// constant of a channel.
__device__ __forceinline__ uint4 load16_plain_if(const void* p, bool yes) {
    uint4 v;
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %5, 0;\n"
        "mov.u32 %0, 0;\nmov.u32 %1, 0;\nmov.u32 %2, 0;\nmov.u32 %3, 0;\n"
        "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((int)yes)
        : "memory");
    return v;
}
__device__ __forceinline__ float load_plain_if(const float* p, bool yes) {
    float v;
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\nmov.f32 %0, 0f00000000;\n@p ld.global.f32 %0, [%1];\n}"
        : "=&f"(v)
        : "l"(p), "r"((int)yes)
        : "memory");
    return v;
}
// (or v stays as it is)
__device__ __forceinline__ void load_plain_onto(float& v, const float* p, bool yes) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\n@p ld.global.f32 %0, [%1];\n}"
                 : "+f"(v)
                 : "l"(p), "r"((int)yes)
                 : "memory");
}
__device__ __forceinline__ float load_if(const float* p, bool yes, float otherwise) {
    float v;
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\nmov.f32 %0, %3;\n@p ld.global.nc.f32 %0, [%1];\n}"
        : "=&f"(v)
        : "l"(p), "r"((int)yes), "f"(otherwise));
    return v;
}

// z * sigmoid(v), v = z (SiLU) or 2 sqrt(2/pi) (z + 0.044715 z^3) (GELU, tanh form:
// (1 + tanh(v/2)) / 2 = sigmoid(v)).  With x = -v log2 e the sigmoid is 1 / (1 + 2^x).
// The special-function unit is what a tile's activation waits for, so four quotients
// share one reciprocal, 1/a = b / (a b) and so on (1.25 instead of 2 operations a
// value).  That holds while the product of four is finite and none is NaN, which
// would reach all four: x at most 30, that is z at least kLeast.  Where a z of the
// warp is below or NaN, each value takes a reciprocal of its own, 0 from 2^x =
// infinity on.  Large negative z then end in -0, and minus infinity in NaN (infinity
// times 0), as the formulas do.  The warp votes on that for a chunk, staying together
// for the loads and stores behind; the shared quotients are formed meanwhile (an
// epilogue warp has one other on its scheduler to hide a vote), and where they do not
// hold the sums are read from tensor memory once more.
template <int kAct>
__device__ __forceinline__ float2 act_exponent(float2 z) {
    if (kAct == NVFP4KV_ACT_SILU)
        return __fmul2_rn(z, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    constexpr float c1 = -1.4426950408889634f * 1.5957691216057308f;
    constexpr float c3 = c1 * 0.044715f;
    return __fmul2_rn(z, __ffma2_rn(__fmul2_rn(z, z), make_float2(c3, c3), make_float2(c1, c1)));
}
// 1 + 2^x of two values
template <int kAct>
__device__ __forceinline__ float2 act_divisor(float2 z) {
    const float2 x = act_exponent<kAct>(z);
    return __fadd2_rn(make_float2(ex2f(x.x), ex2f(x.y)), make_float2(1.0f, 1.0f));
}
__device__ __forceinline__ float rcp_approx(float a) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
// the least of three, or NaN
__device__ __forceinline__ float least_of(float a, float b, float c) {
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Whether all z of the warp, P pairs a lane, are where four may share a reciprocal:
// x(-20.7) = 29.9 and x(-5.5) = 29.8.
template <int kAct, int P>
__device__ __forceinline__ bool warp_shares(const float2 (&z)[P]) {
    constexpr float kLeast = kAct == NVFP4KV_ACT_SILU ? -20.7f : -5.5f;
    float least = 0.0f;
#pragma unroll
    for (int k = 0; k < P; ++k) least = least_of(least, z[k].x, z[k].y);
    return __all_sync(0xFFFFFFFFu, least >= kLeast);
}
template <int kAct, int P>
__device__ __forceinline__ void activate_shared(float2 (&z)[P]) {
#pragma unroll
    for (int k = 0; k < P; k += 2) {
        const float2 d0 = act_divisor<kAct>(z[k]), d1 = act_divisor<kAct>(z[k + 1]);
        const float p0 = d0.x * d0.y, p1 = d1.x * d1.y;
        const float r = rcp_approx(p0 * p1);
        const float r0 = r * p1, r1 = r * p0;       // 1 / p0, 1 / p1
        z[k] = __fmul2_rn(z[k], __fmul2_rn(make_float2(d0.y, d0.x), make_float2(r0, r0)));
        z[k + 1] = __fmul2_rn(z[k + 1], __fmul2_rn(make_float2(d1.y, d1.x), make_float2(r1, r1)));
    }
}
template <int kAct, int P>
__device__ __forceinline__ void activate_each(float2 (&z)[P]) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const float2 d = act_divisor<kAct>(z[k]);
        z[k] = __fmul2_rn(z[k], make_float2(rcp_approx(d.x), rcp_approx(d.y)));
    }
}
// The activation of z, which sums() makes from the accumulators of a chunk.
template <int kAct, int P, class Sums>
__device__ __forceinline__ void activate(float2 (&z)[P], const Sums& sums) {
    if constexpr (kAct != NVFP4KV_ACT_NONE) {
        const bool shares = warp_shares<kAct>(z);
        activate_shared<kAct>(z);
        if (!shares) {
            sums();
            activate_each<kAct>(z);
        }
    }
}

// 2 P tokens' sums of this lane's channel, scaled, with the bias.
template <int P>
__device__ __forceinline__ void channel_sums(uint32_t taddr, float2 (&z)[P], float alpha, float bias) {
    uint32_t v[2 * P];
    if (P == 8) tmem_ld16(taddr, v);
    else if (P == 4) tmem_ld8(taddr, v);
    else tmem_ld4(taddr, v);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < P; ++k)
        z[k] = __ffma2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])),
                          make_float2(alpha, alpha), make_float2(bias, bias));
}

// Walks down the rows of one channel.  Four addresses take turns, each stepping
// four rows, so that a row does not wait for the 64-bit addition of the row
// before; the empty asm keeps the compiler from forming every multiple of the
// row stride ahead of the loops (two registers each).
template <class T>
struct Walk {
    T* p[4];
    __device__ __forceinline__ Walk(T* first, long long ld) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = first + i * ld;
    }
    // the address of row j (rows in order, j known at compile time)
    __device__ __forceinline__ T* row(int j, long long ld) {
        T* r = p[j & 3];
        p[j & 3] += 4 * ld;
        asm("" : "+l"(p[j & 3]));
        return r;
    }
};

// The tensor-memory loads and their wait (and stmatrix, ldmatrix) are instructions
// of a whole warp.  What stands before them may part its lanes (a predicate of a
// lane's channel or token), so each loop below that loads has a __syncwarp() before.

// What an epilogue thread keeps of its tile: its channel n, that channel's
// constants, and where the next token's result and residual are.
struct Channel {
    int n;
    bool stored;             // n < N
    float alpha, bias, gate;
    float* y;
    const float* r;
};

// The residual of the next C tokens, `count` of which exist.
template <int C>
__device__ __forceinline__ void load_residual(const MatmulArgs& a, Walk<const float>& r, float* res, int count) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const float* p = r.row(j, a.ldr);
        load_plain_onto(res[j], p, j < count);
    }
}

// The next C tokens of one channel, `count` of which exist, from their sums in tensor
// memory at taddr and residual res, under ch.gate.
template <int C, int kAct, bool kRes>
__device__ __forceinline__ void finish_tokens(const MatmulArgs& a, uint32_t taddr, const float* res,
                                              const Channel& ch, Walk<float>& y, int count) {
    float2 z[C / 2];
    const auto sums = [&] { channel_sums(taddr, z, ch.alpha, ch.bias); };
    sums();
    activate<kAct>(z, sums);
    const float2 gg = make_float2(ch.gate, ch.gate);
#pragma unroll
    for (int j = 0; j < C; j += 2) {
        float2& f = z[j / 2];
        if (kRes) f = __ffma2_rn(f, gg, make_float2(res[j], res[j + 1]));
        else f = __fmul2_rn(f, gg);
        float* y0 = y.row(j, a.ldy);
        float* y1 = y.row(j + 1, a.ldy);
        if (j < count) *y0 = f.x;
        if (j + 1 < count) *y1 = f.y;
    }
}

// `count` tokens of one channel, accumulators in tensor memory at taddr, all under
// ch.gate; the next 16's residual is on its way meanwhile.  Leaves ch.y and ch.r
// behind the last token.
template <int kAct, bool kRes>
__device__ __forceinline__ void epilogue_run(const MatmulArgs& a, uint32_t taddr, Channel& ch,
                                             int count) {
    float next[kRes ? kChunk : 1] = {};
    Walk<float> y(ch.y, a.ldy);
    Walk<const float> r(ch.r, kRes ? a.ldr : 0);
    ch.y += (size_t)count * a.ldy;
    if (kRes) ch.r += (size_t)count * a.ldr;
    const int here = ch.stored ? 0 : -(1 << 20);      // tokens of no stored channel: none
    if (kRes) load_residual<kChunk>(a, r, next, count + here);
#pragma unroll 1
    for (; count > 0; count -= kChunk, taddr += kChunk) {
        float res[kRes ? kChunk : 1];
        if (kRes) {
#pragma unroll
            for (int j = 0; j < kChunk; ++j) res[j] = next[j];
            load_residual<kChunk>(a, r, next, count - kChunk + here);
        }
        __syncwarp();
        finish_tokens<kChunk, kAct, kRes>(a, taddr, res, ch, y, count + here);
    }
}

// `count` tokens from row m on, their gates looked up one by one.
template <int kAct>
__device__ __forceinline__ void epilogue_gates(const MatmulArgs& a, uint32_t taddr, const Channel& ch,
                                               int m, int count) {
    constexpr int C = 4;
    float* y = ch.y;
    const float* r = ch.r;
#pragma unroll 1
    for (; count > 0; count -= C, taddr += C, m += C) {
        float res[C], g[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const bool here = ch.stored && j < count;
            res[j] = load_plain_if(r + j * a.ldr, here && a.residual);
            g[j] = load_if(a.gate + (size_t)((m + j) / a.rows_per_gate) * a.N + ch.n, here, 0.0f);
        }
        float2 z[2];
        const auto sums = [&] { channel_sums(taddr, z, ch.alpha, ch.bias); };
        __syncwarp();
        sums();
        activate<kAct>(z, sums);
        const float f[C] = {z[0].x, z[0].y, z[1].x, z[1].y};
#pragma unroll
        for (int j = 0; j < C; ++j)
            if (ch.stored && j < count) y[j * a.ldy] = fmaf(f[j], g[j], res[j]);
        y += C * a.ldy;
        r += C * a.ldr;
    }
}

// One warp's share of a tile: `count` tokens from row m on of 32 channels, their
// sums in tensor memory from taddr on.  Gates of 16 rows or more are taken a
// stretch of tokens under one gate at a time.
template <int kAct, bool kGrouped>
__device__ __forceinline__ void epilogue_share(const MatmulArgs& a, uint32_t taddr, int m, int count,
                                               Channel ch) {
    const bool by_row = !kGrouped && a.gate;
    if (by_row && a.rows_per_gate < kChunk) {
        epilogue_gates<kAct>(a, taddr, ch, m, count);
        return;
    }
#pragma unroll 1
    while (count > 0) {
        int n = count;
        if (by_row) {
            const int row = m / a.rows_per_gate;
            n = (int)min((long long)count, (long long)(row + 1) * a.rows_per_gate - m);
            if (ch.stored) ch.gate = __ldg(a.gate + (size_t)row * a.N + ch.n);
        }
        if (a.residual) epilogue_run<kAct, true>(a, taddr, ch, n);
        else epilogue_run<kAct, false>(a, taddr, ch, n);
        taddr += n;
        m += n;
        count -= n;
    }
}

// A bf16 tile's rows in 16-byte pieces (8 channels of one token).  The sums are
// read from tensor memory in the layout of 8 x 8 matrix fragments (thread t of a
// warp: channel t / 4, tokens 2 (t % 4) and the next), so that a pair of tokens
// packs into one register and stmatrix.trans turns fragments into rows of
// channels: per 16 tokens 2 stores of 16 bytes a thread in place of 16 of 2 bytes.
// The residual comes the other way, through ldmatrix.trans.
struct Pieces {
    int n0, lane;            // the warp's first channel
    uint32_t stage;          // its 1 KB of shared memory: 16 tokens x 32 channels
    float bias[4], gate[4];  // of channels n0 + 8 i + lane / 4
    bool here;               // this thread's piece (channels n0 + 8 (lane % 4) ..) exists

    // byte offset of piece p of token t; the swizzle spreads both the 8 tokens of
    // one piece and the 4 pieces of two tokens over all banks
    __device__ __forceinline__ static uint32_t at(int t, int p) {
        return (uint32_t)(t * 64 + ((p ^ (t >> 1)) & 3) * 16);
    }
};

__device__ __forceinline__ void tmem_ld_frag2(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, const uint32_t* r) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Tokens skip .. count - 1 from row m on under pc.gate, accumulators in tensor
// memory at taddr, whole chunks into the tile: the fragments' load takes columns in
// pairs, and an odd column is a misaligned address to it.
template <int kAct, bool kRes>
__device__ __forceinline__ void epilogue_pieces(const MatmulArgs& a, uint32_t taddr, const Pieces& pc,
                                                int m, int skip, int count, float alpha) {
    const int tok = pc.lane >> 2, piece = pc.lane & 3;
    const size_t first = (size_t)(m + tok), col = (size_t)(pc.n0 + 8 * piece);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.Y) + first * a.ldy + col;
    const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(a.residual) + first * a.ldr + col;
    // the rows that this thread hands to stmatrix / ldmatrix (matrix lane / 8 =
    // channels 8 (lane / 8) .., token lane % 8), and its own pieces
    const uint32_t frag = pc.stage + Pieces::at(pc.lane & 7, pc.lane >> 3);
    const uint32_t own = pc.stage + Pieces::at(tok, piece);
    constexpr uint32_t kHalf = 8 * 64;       // tokens 8 .. 15 (the swizzle repeats)
    uint4 next[2];
    auto mine = [&](int t) { return pc.here && t >= skip && t < count; };
    auto load = [&](int ahead) {
        next[0] = load16_plain_if(r, mine(tok + ahead));
        next[1] = load16_plain_if(r + 8 * a.ldr, mine(tok + ahead + 8));
        r += kChunk * a.ldr;
    };
    if (kRes) load(0);
#pragma unroll 1
    for (; count > 0; count -= kChunk, skip -= kChunk, taddr += kChunk) {
        uint32_t v[16], res[8];
        const auto load_sums = [&] {
            tmem_ld_frag2(taddr, v);
            tmem_ld_frag2(taddr + (16u << 16), v + 8);
        };
        __syncwarp();                        // the last chunk's pieces are read and stored
        load_sums();
        if (kRes) {
            sts16(own, next[0]);
            sts16(own + kHalf, next[1]);
            load(kChunk);
            __syncwarp();
            ldmatrix4_trans(frag, res);
            ldmatrix4_trans(frag + kHalf, res + 4);
            __syncwarp();
        }
        float2 z[8];                         // tokens 8 j .., channels 8 i ..: z[4 j + i]
        const auto scaled = [&] {
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = k & 3;
                const uint32_t* q = v + 8 * (i >> 1) + 4 * (k >> 2) + 2 * (i & 1);
                z[k] = __ffma2_rn(make_float2(__uint_as_float(q[0]), __uint_as_float(q[1])),
                                  make_float2(alpha, alpha), make_float2(pc.bias[i], pc.bias[i]));
            }
        };
        scaled();
        activate<kAct>(z, [&] {
            load_sums();
            scaled();
        });
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2& f = z[4 * j + i];
                const float2 g = make_float2(pc.gate[i], pc.gate[i]);
                if (kRes) {
                    const uint32_t w = res[4 * j + i];
                    f = __ffma2_rn(f, g, make_float2(__uint_as_float(w << 16),
                                                     __uint_as_float(w & 0xFFFF0000u)));
                } else {
                    f = __fmul2_rn(f, g);
                }
                const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
                p[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            stmatrix4_trans(frag + j * kHalf, p);
        }
        __syncwarp();
        if (mine(tok)) *reinterpret_cast<uint4*>(y) = lds16(own);
        if (mine(tok + 8)) *reinterpret_cast<uint4*>(y + 8 * a.ldy) = lds16(own + kHalf);
        y += kChunk * a.ldy;
    }
}

// One warp's share of a bf16 tile in pieces: stretches of tokens under one gate, a
// chunk that two of them share once for each.
template <int kAct, bool kGrouped>
__device__ __forceinline__ void epilogue_pieces_share(const MatmulArgs& a, uint32_t taddr, Pieces& pc,
                                                      int m, int count, float alpha) {
    const bool by_row = !kGrouped && a.gate;
    int skip = 0;                            // tokens of the chunk at m that are done
#pragma unroll 1
    while (skip < count) {
        int n = count;
        if (by_row) {
            const int row = (m + skip) / a.rows_per_gate;
            n = (int)min((long long)count, (long long)(row + 1) * a.rows_per_gate - m);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = pc.n0 + 8 * i + (pc.lane >> 2);
                pc.gate[i] = load_if(a.gate + (size_t)row * a.N + c, c < a.N, 0.0f);
            }
        }
        if (a.residual) epilogue_pieces<kAct, true>(a, taddr, pc, m, skip, n, alpha);
        else epilogue_pieces<kAct, false>(a, taddr, pc, m, skip, n, alpha);
        const int whole = n / kChunk * kChunk;
        taddr += whole;
        m += whole;
        count -= whole;
        skip = n - whole;
    }
}

// A bf16 tile whose rows are no whole pieces, or whose gates change within a
// chunk, by way of fp32 rows: 8 tokens at a time, sums with a thread a channel
// (bias, activation and gate there), then through shared memory to a thread for 4
// channels of one token, which adds the residual, rounds and stores: 8 bytes
// at once where `vec`, else element by element.
__device__ __forceinline__ void unpack4(const uint2& v, float* f) {
    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ uint2 pack4(const float* f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Tokens skip .. count - 1 from row m on, accumulators in tensor memory at taddr (a
// multiple of 8 tokens into the tile).  gate: of this lane's channel n0 + lane;
// kGates: looked up for each token instead.
template <int kAct, bool kRes, bool kGates>
__device__ __forceinline__ void epilogue_rows(const MatmulArgs& a, uint32_t taddr, int n0, int lane,
                                              float* stage, int m, int skip, int count, float alpha,
                                              float bias, float gate, bool vec) {
    using T = __nv_bfloat16;
    constexpr int C = 8;
    const int tok = lane >> 3, col = 4 * (lane & 7);
    const int here = min(4, a.N - n0 - col);             // channels of this thread that exist
    T* y = static_cast<T*>(a.Y) + (size_t)(m + tok) * a.ldy + n0 + col;
    const T* r = static_cast<const T*>(a.residual) + (size_t)(m + tok) * a.ldr + n0 + col;
    uint2 next[2];
    auto is_mine = [&](int t) { return t >= skip && t < count && here > 0; };
    auto load = [&](int ahead) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (is_mine(tok + ahead + 4 * h)) next[h] = *reinterpret_cast<const uint2*>(r + 4 * h * a.ldr);
        r += C * a.ldr;
    };
    if (kRes && vec) load(0);
#pragma unroll 1
    for (; count > 0; count -= C, skip -= C, taddr += C) {
        float2 z[C / 2];
        const auto sums = [&] { channel_sums(taddr, z, alpha, bias); };
        __syncwarp();                        // the last tokens' rows are read and stored
        sums();
        activate<kAct>(z, sums);
#pragma unroll
        for (int k = 0; k < C / 2; ++k) {
            z[k] = __fmul2_rn(z[k], make_float2(gate, gate));
            stage[2 * k * 32 + lane] = z[k].x;
            stage[(2 * k + 1) * 32 + lane] = z[k].y;
        }
        __syncwarp();
        uint2 now[2];
        if (kRes && vec) {
            now[0] = next[0];
            now[1] = next[1];
            load(C);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool mine = is_mine(tok + 4 * h);
            const float4 q = *reinterpret_cast<const float4*>(stage + (tok + 4 * h) * 32 + col);
            float f[4] = {q.x, q.y, q.z, q.w};
            if (kGates && mine) {
                const float* g = a.gate + (size_t)((m + tok + 4 * h) / a.rows_per_gate) * a.N + n0 + col;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < here) f[i] *= __ldg(g + i);
            }
            if (vec) {
                if (kRes) {
                    float w[4];
                    unpack4(now[h], w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] += w[i];
                }
                if (mine) *reinterpret_cast<uint2*>(y + 4 * h * a.ldy) = pack4(f);
            } else if (mine) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < here) {
                        if (kRes) f[i] += __bfloat162float(r[4 * h * a.ldr + i]);
                        y[4 * h * a.ldy + i] = __float2bfloat16_rn(f[i]);
                    }
            }
        }
        y += C * a.ldy;
        m += C;
        if (!vec) r += C * a.ldr;
    }
}

// One warp's share of a tile in fp32 rows: stretches of tokens under one gate, or
// all of them with a gate looked up for each where a gate holds for less than 16.
template <int kAct, bool kGrouped>
__device__ __forceinline__ void epilogue_rows_share(const MatmulArgs& a, uint32_t taddr, int n0, int lane,
                                                    float* stage, int m, int count, float alpha,
                                                    float bias, float gate, bool vec) {
    const bool by_row = !kGrouped && a.gate;
    if (by_row && a.rows_per_gate < kChunk) {
        if (a.residual)
            epilogue_rows<kAct, true, true>(a, taddr, n0, lane, stage, m, 0, count, alpha, bias, 1.0f,
                                            vec);
        else
            epilogue_rows<kAct, false, true>(a, taddr, n0, lane, stage, m, 0, count, alpha, bias, 1.0f,
                                             vec);
        return;
    }
    constexpr int C = 8;
    int skip = 0;                            // tokens of the 8 at m that are done
#pragma unroll 1
    while (skip < count) {
        int n = count;
        if (by_row) {
            const int row = (m + skip) / a.rows_per_gate;
            n = (int)min((long long)count, (long long)(row + 1) * a.rows_per_gate - m);
            gate = n0 + lane < a.N ? __ldg(a.gate + (size_t)row * a.N + n0 + lane) : 0.0f;
        }
        if (a.residual)
            epilogue_rows<kAct, true, false>(a, taddr, n0, lane, stage, m, skip, n, alpha, bias, gate, vec);
        else
            epilogue_rows<kAct, false, false>(a, taddr, n0, lane, stage, m, skip, n, alpha, bias, gate, vec);
        const int whole = n / C * C;
        taddr += whole;
        m += whole;
        count -= whole;
        skip = n - whole;
    }
}

struct TileAt {
    int e, n0, m0, m_end;    // expert, first channel, rows [m0, m_end)
    int tokens;              // m_end - m0 rounded up to 16: the MMA's N
};

// Rows of a tile of a group of `rows` > 0: as few tiles as TN allows, of one size,
// a multiple of 16 (the last may be shorter).
template <int TN>
__host__ __device__ __forceinline__ int tile_rows(int rows) {
    const int count = (rows + TN - 1) / TN;
    return ((rows + count - 1) / count + 15) / 16 * 16;
}

template <int TN, int G, bool kGrouped>
struct Tiles {
    const MatmulArgs& a;
    const int* s_off;        // grouped: row offsets, first tiles and tile rows of the groups
    const int* s_tile;
    const int* s_size;
    int n_tiles, e, rank, size;
    __device__ Tiles(const MatmulArgs& args, const int* off, const int* tile, const int* sizes,
                     int rank_)
        : a(args), s_off(off), s_tile(tile), s_size(sizes), e(0), rank(rank_) {
        n_tiles = (a.N + kTileN * G - 1) / (kTileN * G);
        size = kGrouped ? 0 : tile_rows<TN>(a.M);
    }
    __device__ int total() const {
        return kGrouped ? s_tile[a.E] : ((a.M + TN - 1) / TN) * n_tiles;
    }
    // t grows from call to call
    __device__ TileAt at(int t) {
        TileAt r;
        int row0 = 0, m_end = a.M;        // the group's rows
        if (kGrouped) {
            while (s_tile[e + 1] <= t) ++e;
            t -= s_tile[e];
            row0 = s_off[e];
            m_end = s_off[e + 1];
            size = s_size[e];
        }
        const int mt = t / n_tiles;
        r.e = e;
        r.n0 = ((t - mt * n_tiles) * G + rank) * kTileN;   // this CTA's channels
        r.m0 = row0 + mt * size;
        r.m_end = min(m_end, r.m0 + size);
        r.tokens = (r.m_end - r.m0 + 15) / 16 * 16;
        return r;
    }
};

template <int TN, int G, bool kGrouped, bool kF32>
__global__ void __launch_bounds__(kThreadsMM, 1)
matmul_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
              const __grid_constant__ MatmulArgs a) {
    using S = Shape<TN, G>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ MMShared sh;
    __shared__ int s_off[kGrouped ? kMaxExperts + 1 : 1];
    __shared__ int s_tile[kGrouped ? kMaxExperts + 1 : 1];
    __shared__ int s_size[kGrouped ? kMaxExperts : 1];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &sh.abort;
    // a pair is a cluster of two CTAs; rank 0 leads (issues its MMAs)
    const int rank = G == 1 ? 0 : (int)(blockIdx.x & 1u);
    const int first_tile = blockIdx.x / G, stride = gridDim.x / G;
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);

    if (warp == kMmaWarp) {
        if (G == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&sh.tmem_base)),
                         "r"(kColsMM));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&sh.tmem_base)),
                         "r"(kColsMM));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        }
    }
    if (tid == 0) {
        sh.abort = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_u32(&sh.tma_full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.sf_full[i]), kScaleWarps + (G - 1));
            mbar_init(smem_u32(&sh.sf_own[i]), kScaleWarps);
            mbar_init(smem_u32(&sh.sf_empty[i]), 1);
            mbar_init(smem_u32(&sh.acc_full[i]), 1);
            mbar_init(smem_u32(&sh.acc_free[i]), (kEpiWarps + (a.residual ? 1 : 0)) * G);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (kGrouped && warp == 0) {
        // tile count prefix over the experts; offsets that decrease or leave
        // [0, M] are reported and nothing is computed
        const int nt = (a.N + kTileN * G - 1) / (kTileN * G);
        int carry = 0;
        bool bad = false;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            int cnt = 0;
            if (e < a.E) {
                const int o0 = a.offsets[e], o1 = a.offsets[e + 1];
                const bool fits = o0 >= 0 && o1 >= o0 && o1 <= a.M;
                const int rows = fits ? o1 - o0 : 0;
                bad |= !fits;
                s_off[e] = o0;
                if (e == a.E - 1) s_off[a.E] = o1;
                cnt = (rows + TN - 1) / TN * nt;
                s_size[e] = rows > 0 ? tile_rows<TN>(rows) : 0;
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
        __syncwarp();            // the last group's lane has written s_tile[E]
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
    if (G == 2) cluster_sync();      // both CTAs' barriers are ready
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    Tiles<TN, G, kGrouped> tiles(a, s_off, s_tile, s_size, rank);
    const int total = tiles.total();
    const int steps = (a.K + kStageK - 1) / kStageK;
    const int turns = (steps + kTurn - 1) / kTurn;
    const int kbytes = a.K / 16;
    uint8_t* sf_base = base + (size_t)S::kStages * S::kStage;
    uint8_t* epi_base = sf_base + 2 * S::kSfStage;

    if (warp < kEpiWarp0)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    else
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    if (warp < kTmaWarp) {
        // ------------------------------------------------------------ block scales
        // Per turn, 4 steps (64 scale bytes a row) of every 128-row group.  Unit u
        // of a warp: rows 32 g + r of group u / 4 (0: weights), g = lane % 4,
        // r = 8 (u % 4) + 2 warp + lane / 16, bytes 16 q .. 16 q + 15 of the
        // turn's 64, q = lane / 4 % 4: a row's 64 bytes are read together, and
        // the words stored together are of 4 row groups and 2 rows.
        constexpr int kUnits = S::kGroups * 4;
        const bool withhold = blockIdx.x == 0 && warp == 0 && (a.ctl->test_flags & 1u) != 0u;
        const int g = lane & 3, q = (lane >> 2) & 3;
        const int r = 2 * warp + (lane >> 4);
        uint32_t w[kUnits][5];        // a unit's words, and the half word it ends in
        uint32_t odds = 0;            // units whose rows begin in mid-word
        int turn_left = 0;            // bytes of this lane's 16 that a row has
        const bool wide = kbytes % 16 == 0 && a.x_shift == 0;
        auto fetch = [&](const TileAt& at, int turn) {
            const int kb = turn * 64 + q * 16;
            const int nw = at.n0 + 32 * g + r, mx = at.m0 + 32 * g + r;
            const uint8_t* wp = a.w_scales + (size_t)at.e * a.w_scale_rows * kbytes + kb;
            const uint8_t* xp = a.x_scales + kb;
            if (wide) {
                const int n_end = kb < kbytes ? a.N : 0;
                const int m_end = kb < kbytes ? at.m_end : 0;
                // rows 8 apart; in tiles rows 16 apart have scale rows 1 apart
                // (n0 is a multiple of 16)
                const uint8_t* p = wp + (size_t)(nw >> a.w_shift) * kbytes;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    put_words(w[u], load16_if(p, nw + 8 * u < n_end));
                    p += a.w_shift ? (u & 1) * kbytes : 8 * kbytes;
                }
                p = xp + (size_t)mx * kbytes;
#pragma unroll
                for (int u = 4; u < kUnits; ++u) {
                    put_words(w[u], load16_if(p, mx + 8 * (u & 3) + 128 * (u / 4 - 1) < m_end));
                    p += (u & 3) == 3 ? 104 * kbytes : 8 * kbytes;
                }
            } else {
                // K no multiple of 256 (or X in tiles): rows at even addresses; by
                // whole words where K is a multiple of 64
                odds = 0;
                turn_left = max(0, min(16, kbytes - kb));
                auto unit = [&](int u, int& left) {
                    const int i = (u < 4 ? nw : mx + 128 * (u / 4 - 1)) + 8 * (u & 3);
                    left = i < (u < 4 ? a.N : at.m_end) ? turn_left : 0;
                    return (u < 4 ? wp : xp) +
                           (size_t)(i >> (u < 4 ? a.w_shift : a.x_shift)) * kbytes;
                };
                int left;
                if (kbytes % 4 == 0) {
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) {
                        const uint8_t* p = unit(u, left);
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[u][j] = load4_if(p + 4 * j, left > 4 * j);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) {
                        const uint8_t* p = unit(u, left);
                        // the aligned words that the row fills, and the half word
                        // that it may end in (at most one); nothing behind the row
                        // is read
                        const int odd = (int)(reinterpret_cast<uintptr_t>(p) >> 1 & 1);
                        odds |= (uint32_t)odd << u;
                        p -= 2 * odd;
                        const int bytes = left > 0 ? left + 2 * odd : 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[u][j] = load4_if(p + 4 * j, bytes >= 4 * j + 4);
                        w[u][4] = load2_if(p + (bytes & ~3), (bytes & 2) != 0);
                    }
                }
            }
        };
        auto put = [&](uint8_t* sf) {
            uint8_t* line = sf + 4 * q * kSfBlock + r * 16 + g * 4;
            auto at = [&](int u, int j) {
                return reinterpret_cast<uint32_t*>(line + (u / 4) * kSfGroup + (u & 3) * 128 +
                                                   j * kSfBlock);
            };
            if (kbytes % 4 == 0) {
#pragma unroll
                for (int u = 0; u < kUnits; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) *at(u, j) = w[u][j];
            } else {
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const int odd = (int)(odds >> u & 1u), bytes = turn_left + 2 * odd;
                    const int half = (bytes & 2) ? bytes >> 2 : 5;     // the half word's place
                    uint32_t v[5];
#pragma unroll
                    for (int j = 0; j < 5; ++j) v[j] = half == j ? w[u][4] : j < 4 ? w[u][j] : 0u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) *at(u, j) = __funnelshift_r(v[j], v[j + 1], 16 * odd);
                }
            }
        };
        int it = 0;
        bool ok = true;
        if (first_tile < total) fetch(tiles.at(first_tile), 0);
        for (int t = first_tile; t < total && ok; t += stride) {
            const TileAt at = tiles.at(t);
            for (int turn = 0; turn < turns; ++turn, ++it) {
                const int st = it & 1;
                ok = wait_or_abort_m(smem_u32(&sh.sf_empty[st]), (uint32_t)(((it >> 1) & 1) ^ 1), abort,
                                     a.ctl, 60u, it);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                put(sf_base + st * S::kSfStage);
                fence_async_smem();
                __syncwarp();
                if (lane == 0 && !(withhold && it == 0))
                    mbar_arrive(smem_u32(rank == 0 ? &sh.sf_full[st] : &sh.sf_own[st]));
                if (turn + 1 < turns) fetch(at, turn + 1);
                else if (t + stride < total) fetch(tiles.at(t + stride), 0);
            }
        }
        // the last turns are signalled as done here before the CTA leaves (the
        // leader's commits arrive in both)
        for (int i = max(it - 2, 0); i < it && ok; ++i)
            ok = wait_or_abort_m(smem_u32(&sh.sf_empty[i & 1]), (uint32_t)((i >> 1) & 1), abort, a.ctl,
                                 60u, i);
    } else if (warp >= kEpiWarp0) {
        // ------------------------------------------------------------ epilogue
        // warp = lane quarter (warp % 4) of one part of the tile's tokens
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        uint8_t* stage = epi_base + (warp - kEpiWarp0) * kEpiBytes;
        // bf16 rows go in whole pieces of 8 elements where a gate holds for at
        // least a chunk, else in pieces of 4 or by element
        const uintptr_t align = reinterpret_cast<uintptr_t>(a.Y) | (uintptr_t)(a.ldy * 2) |
                                (a.residual ? reinterpret_cast<uintptr_t>(a.residual) |
                                                  (uintptr_t)(a.ldr * 2)
                                            : 0);
        const bool vec = align % 8 == 0 && a.N % 4 == 0;
        const bool pieces = align % 16 == 0 && a.N % 8 == 0 &&
                            (kGrouped || !a.gate || a.rows_per_gate >= kChunk);
        // a tile's place and its channel's constants, loaded a tile ahead
        struct {
            TileAt at;
            float scale, bias, gate;
        } next = {};
        const float x_scale = __ldg(a.x_scale);
        auto look = [&](int t) {
            next.at = tiles.at(t);
            const int n = next.at.n0 + (warp & 3) * 32 + lane;
            const size_t en = (size_t)next.at.e * a.N + n;
            next.scale = __ldg(a.w_scale + next.at.e);
            next.bias = load_if(a.bias + en, a.bias && n < a.N, 0.0f);
            next.gate = load_if(a.gate + en, a.gate && kGrouped && n < a.N, 1.0f);
        };
        if (first_tile < total) look(first_tile);
        int i = 0;
        for (int t = first_tile; t < total; t += stride, ++i) {
            const TileAt at = next.at;
            const float alpha = x_scale * next.scale, bias = next.bias, gate = next.gate;
            const int buf = i & 1;
            constexpr int kParts = kEpiWarps / 4;
            const int part = ((at.tokens + kParts - 1) / kParts + kChunk - 1) / kChunk * kChunk;
            const int first = (warp - kEpiWarp0) / 4 * part;
            const int m = at.m0 + first;
            const int count = min(part, at.m_end - m);
            const int n0 = at.n0 + (warp & 3) * 32;
            const bool stored = n0 + lane < a.N;
            if (t + stride < total) look(t + stride);
            const bool got = wait_or_abort_m(smem_u32(&sh.acc_full[buf]), (uint32_t)((i >> 1) & 1),
                                             abort, a.ctl, 61u, i);
            if (!__all_sync(0xFFFFFFFFu, got)) break;
            tc_fence_after();
            const uint32_t ta = tmem + lane_base + (uint32_t)(buf * TN + first);
            auto finish = [&](auto act) {
                constexpr int kAct = decltype(act)::value;
                if constexpr (kF32) {
                    Channel ch;
                    ch.n = n0 + lane;
                    ch.stored = stored;
                    ch.alpha = alpha;
                    ch.bias = bias;
                    ch.gate = gate;
                    ch.y = static_cast<float*>(a.Y) + (size_t)m * a.ldy + ch.n;
                    ch.r = static_cast<const float*>(a.residual) + (size_t)m * a.ldr + ch.n;
                    epilogue_share<kAct, kGrouped>(a, ta, m, count, ch);
                } else if (pieces) {
                    Pieces pc;
                    pc.n0 = n0;
                    pc.lane = lane;
                    pc.stage = smem_u32(stage);
                    pc.here = n0 + 8 * (lane & 3) < a.N;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        pc.bias[k] = __shfl_sync(0xFFFFFFFFu, bias, 8 * k + (lane >> 2));
                        pc.gate[k] = __shfl_sync(0xFFFFFFFFu, gate, 8 * k + (lane >> 2));
                    }
                    epilogue_pieces_share<kAct, kGrouped>(a, ta, pc, m, count, alpha);
                } else {
                    epilogue_rows_share<kAct, kGrouped>(a, ta, n0, lane, reinterpret_cast<float*>(stage), m,
                                                        count, alpha, bias, gate, vec);
                }
            };
            if (a.act == NVFP4KV_ACT_GELU_TANH) finish(IntC<NVFP4KV_ACT_GELU_TANH>());
            else if (a.act == NVFP4KV_ACT_SILU) finish(IntC<NVFP4KV_ACT_SILU>());
            else finish(IntC<NVFP4KV_ACT_NONE>());
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader<G>(smem_u32(&sh.acc_free[buf]));
        }
    } else if (warp == kTmaWarp) {
        // ------------------------------------------------------------ code tiles
        if (elect_one()) {
            Ring<S::kStages> ring;
            int it = 0;
            bool ok = true;
            const uint32_t stage0 = smem_u32(base);
            for (int t = first_tile; t < total && ok; t += stride) {
                const TileAt at = tiles.at(t);
                // this CTA's share of the token rows, a box at a time
                const int m0 = at.m0 + rank * (at.tokens / G);
                const int boxes = (at.tokens / G + S::kBox - 1) / S::kBox;
                for (int s = 0; s < steps; ++s, ++it, ring.next()) {
                    // (the first pass over the ring finds the phase before the first done)
                    ok = wait_or_abort_m(smem_u32(&sh.empty[ring.at]), ring.phase ^ 1u, abort, a.ctl,
                                         62u, it);
                    if (!ok) break;
                    const uint32_t dst = stage0 + (uint32_t)ring.at * S::kStage;
                    // the leader's barrier counts both CTAs' bytes
                    uint32_t bar = smem_u32(&sh.tma_full[ring.at]);
                    if (rank == 0) mbar_expect_tx(bar, (uint32_t)(G * (kATile + boxes * S::kBox * 128)));
                    if (G == 2) bar = leader_addr(bar);
                    tma_load_3d<G>(dst, &map_w, s * 128, at.n0, at.e, bar);
#pragma unroll
                    for (int i = 0; i < TN / G / S::kBox; ++i)
                        if (i < boxes)
                            tma_load_3d<G>(dst + kATile + i * S::kBox * 128, &map_x, s * 128,
                                           m0 + i * S::kBox, 0, bar);
                }
            }
            // the last uses of the stages are signalled here before the CTA leaves
            for (int i = min(it, S::kStages); i > 0 && ok; --i, ring.next()) {
                if (it < S::kStages && i == it) ring = Ring<S::kStages>();
                ok = wait_or_abort_m(smem_u32(&sh.empty[ring.at]),
                                     it < S::kStages ? 0u : ring.phase ^ 1u, abort, a.ctl, 66u, i);
            }
            if (!ok) {
                // after a wait that gave up: the loads in flight have landed long
                // before this ends (a pair's are counted in the other CTA)
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < kLandNs) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == kPrefetchWarp && a.residual) {
        // ------------------------------------------------------------ residual
        // Each tile's residual into L2 while its sums are formed: the epilogue
        // then waits for L2, not for HBM.  A step ahead of the epilogue, which
        // it may not outrun (it takes part in freeing the accumulators).
        constexpr int kSize = kF32 ? 4 : 2;
        const char* res = static_cast<const char*>(a.residual);
        int i = 0;
        for (int t = first_tile; t < total; t += stride, ++i) {
            const TileAt at = tiles.at(t);
            const int bytes = min(kTileN, a.N - at.n0) * kSize;
            constexpr int kLines = kTileN * kSize / 128;      // lanes of a row
            for (int r = lane / kLines; r < at.m_end - at.m0; r += 32 / kLines) {
                const int b = lane % kLines * 128;
                if (b < bytes)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(
                        res + ((size_t)(at.m0 + r) * a.ldr + at.n0) * kSize + b));
            }
            if (i > 0) {
                const bool got = wait_or_abort_m(smem_u32(&sh.acc_full[(i - 1) & 1]),
                                                 (uint32_t)(((i - 1) >> 1) & 1), abort, a.ctl, 67u, i);
                if (!__all_sync(0xFFFFFFFFu, got)) break;
                if (lane == 0) arrive_leader<G>(smem_u32(&sh.acc_free[(i - 1) & 1]));
            }
        }
        // (no arrival for the last tile: no tile waits for its accumulator, and
        // before its sums are full the arrival would count for the tile two before)
    } else if (warp == kMmaWarp && rank == 0) {
        // ------------------------------------------------------------ MMA issue
        // One elected lane walks the steps.  (elect.sync, not lane == 0: knowing
        // the branch to be one thread, the compiler issues the tensor-core
        // instructions straight from uniform registers.)
        if (elect_one()) {
            Ring<S::kStages> ring;
            Ring<2> turn, acc;
            const uint32_t stage0 = smem_u32(base), sf0 = smem_u32(sf_base);
            bool ok = true;
            for (int t = first_tile; t < total && ok; t += stride, acc.next()) {
                // (the first use of an accumulator finds the phase before the first done)
                ok = wait_or_abort_m(smem_u32(&sh.acc_free[acc.at]), acc.phase ^ 1u, abort, a.ctl, 63u,
                                     t);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)acc.at * TN;
                const uint32_t idesc = umma_idesc_scaled(G * kTileN, (uint32_t)tiles.at(t).tokens);
                for (int s = 0; s < steps; s += kTurn, turn.next()) {
                    ok = wait_or_abort_m<(G > 1)>(smem_u32(&sh.sf_full[turn.at]), turn.phase, abort,
                                                  a.ctl, 64u, s);
                    if (!ok) break;
                    const uint32_t sf = sf0 + (uint32_t)turn.at * S::kSfStage;
                    const int n = min(kTurn, steps - s);
#pragma unroll 1
                    for (int k = 0; k < n; ++k, ring.next()) {
                        ok = wait_or_abort_m(smem_u32(&sh.tma_full[ring.at]), ring.phase, abort, a.ctl,
                                             65u, s);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t sa = stage0 + (uint32_t)ring.at * S::kStage;
                        const uint64_t da = umma_desc(sa, 16, 1024);
                        const uint64_t db = umma_desc(sa + kATile, 16, 1024);
                        const uint64_t ds = umma_desc_noswizzle(sf + k * 4 * kSfBlock, 16, 128);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            tmem_cp_scales<G>(tmem + S::kColSFA + 4u * j,
                                              ds + (uint64_t)((kSfBlock * j) >> 4));
#pragma unroll
                            for (int q = 1; q < S::kGroups; ++q)
                                tmem_cp_scales<G>(tmem + S::kColSFB + 8u * j + 4u * (q - 1),
                                                  ds + (uint64_t)((kSfGroup * q + kSfBlock * j) >> 4));
                        }
                        // the turn's scales are in tensor memory once its last copies are
                        // done, a step before its last MMAs
                        if (k == n - 1) commit_all<G>(smem_u32(&sh.sf_empty[turn.at]));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_scaled<G>(d, da + 2u * j, db + 2u * j, idesc, (s | k | j) ? 1u : 0u,
                                          tmem + S::kColSFA + 4u * j, tmem + S::kColSFB + 8u * j);
                        commit_all<G>(smem_u32(&sh.empty[ring.at]));
                    }
                    if (!ok) break;
                }
                if (ok) commit_all<G>(smem_u32(&sh.acc_full[acc.at]));
            }
            commit_own<G>(smem_u32(&sh.drain));
            mbar_wait(smem_u32(&sh.drain), 0u);
        }
        __syncwarp();
    } else if (G == 2 && warp == kMmaWarp) {
        // ------------------------------------------------------------ scales of a pair
        // The leader's copies read the second CTA's scales in that CTA's shared
        // memory, so they are handed over at cluster scope, once a turn.  This warp
        // releases them, since a release waits for what its warp has in flight (the
        // scale warps: the next turn's loads; [7040, 8192] x [2048, 8192] took 77 us
        // with the release in those, 65 to 67 so).
        if (elect_one()) {
            Ring<2> turn;
            bool ok = true;
            for (int t = first_tile; t < total && ok; t += stride)
                for (int k = 0; k < turns && ok; ++k, turn.next()) {
                    ok = wait_or_abort_m(smem_u32(&sh.sf_own[turn.at]), turn.phase, abort, a.ctl, 64u, k);
                    if (ok) mbar_arrive_release_cluster(leader_addr(smem_u32(&sh.sf_full[turn.at])));
                }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (G == 2) cluster_sync();      // neither CTA leaves while the other may signal it
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        if (G == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(kColsMM));
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
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
template <int TN, int G, bool kGrouped, bool kF32>
bool configure(int dev) {
    static std::atomic<bool> done[kMaxDevices];
    if (done[dev].load(std::memory_order_relaxed)) return true;
    if (cudaFuncSetAttribute(matmul_kernel<TN, G, kGrouped, kF32>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Shape<TN, G>::kSmem) != cudaSuccess)
        return false;
    done[dev].store(true, std::memory_order_relaxed);
    return true;
}

template <int TN, int G, bool kGrouped, bool kF32>
nvfp4kv_status launch_tn(const MatmulArgs& a, const void* w_codes, const void* x_codes, int dev,
                         int sms, cudaStream_t stream) {
    CUtensorMap map_w, map_x;
    if (!make_map(&map_w, w_codes, a.K, a.N, kGrouped ? a.E : 1, kTileN) ||
        !make_map(&map_x, x_codes, a.K, a.M, 1, Shape<TN, G>::kBox) || !configure<TN, G, kGrouped, kF32>(dev))
        return NVFP4KV_ERR_CUDA;
    const long long n_tiles = (a.N + kTileN * G - 1) / (kTileN * G);
    // grouped: at most one more token tile per expert than the rows fill
    const long long most = n_tiles * ((a.M + TN - 1) / TN + (kGrouped ? a.E : 0));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(G * (unsigned)(most < sms / G ? most : sms / G));
    cfg.blockDim = dim3(kThreadsMM);
    cfg.dynamicSmemBytes = Shape<TN, G>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = G;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = G > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, matmul_kernel<TN, G, kGrouped, kF32>, map_w, map_x, a) ==
                   cudaSuccess
               ? NVFP4KV_OK
               : NVFP4KV_ERR_CUDA;
}

// Tokens a tile (TN) for this product.  Wide tiles read each weight for more tokens,
// and a pair of CTAs shares them ([7040, 8192] x [2048, 8192] took 91, 70, 66 and 69
// us with 64, 128, 192 and 224 tokens, [7266, 2048] over two [2048, 2048] 39, 32, 31
// and 30); narrow ones give more CTAs work and leave a shorter epilogue (about 0.8 us
// and 25 ns a token) after the last MMA: [880, 2048] x [2048, 2048] took 11.5, 8.2,
// 6.8, 9.0 and 9.6 us with 32 to 224 tokens, [200, 4096] x [4096, 4096] 10.8, 8.2, 8.3,
// 10.4 and 11.4.  A pair costs 1.8 us more to begin and 0.08 us more a step of 256
// along k, which only more than 128 tokens a tile make up for: one row with K = 512,
// 2048 and 8192 took 4.1, 5.4 and 9.5 us on single CTAs and 5.9, 7.1 and 13.1 on
// pairs.  The rule adds these up in ns, as they are on a full device, and takes the
// least.  A grouped product's group sizes are not known here: their mean stands for
// all.
int choose_tile(int M, int N, int K, int E, int sms) {
    const double steps = (K + kStageK - 1) / kStageK;
    int best = 0;
    double least = 0.0;
    for (const int tn : {32, 64, 128, 192, 224}) {
        const int g = tn > 128 ? 2 : 1;
        const double per = (double)M / E;
        // groups of all sizes: half a tile each goes to the ragged end
        const double count = E == 1 ? std::ceil(per / tn) : std::max(1.0, per / tn + 0.5);
        const double size = std::ceil(per / count / 16.0) * 16.0;
        if (g == 2 && size <= 128.0) continue;
        const double tiles = count * E * ((N + kTileN * g - 1) / (kTileN * g));
        double waves = tiles / (sms / g);
        if (E <= 4 || waves < 1.0) waves = std::ceil(waves);   // many groups even out
        const double sums = steps * (g == 1 ? 250.0 + 1.1 * size : 170.0 + 1.6 * size);
        const double epilogue = 800.0 + 25.0 * size;
        const double cost = (g == 1 ? 0.0 : 1200.0) + sums + epilogue +
                            (waves - 1.0) * std::max(sums, epilogue);
        if (best == 0 || cost < least) {
            best = tn;
            least = cost;
        }
    }
    return best;
}

template <bool kGrouped, bool kF32>
nvfp4kv_status launch_any(const MatmulArgs& a, const void* w_codes, const void* x_codes,
                          cudaStream_t stream) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return NVFP4KV_ERR_CUDA;
    const int sms = sm_count_of(dev);
    if (sms < 2) return NVFP4KV_ERR_CUDA;
    switch (choose_tile(a.M, a.N, a.K, a.E, sms)) {
        case 32: return launch_tn<32, 1, kGrouped, kF32>(a, w_codes, x_codes, dev, sms, stream);
        case 64: return launch_tn<64, 1, kGrouped, kF32>(a, w_codes, x_codes, dev, sms, stream);
        case 128: return launch_tn<128, 1, kGrouped, kF32>(a, w_codes, x_codes, dev, sms, stream);
        case 192: return launch_tn<192, 2, kGrouped, kF32>(a, w_codes, x_codes, dev, sms, stream);
        default: return launch_tn<224, 2, kGrouped, kF32>(a, w_codes, x_codes, dev, sms, stream);
    }
}

}  // namespace

int matmul_tile(int M, int N, int K, int E, int sms) { return choose_tile(M, N, K, E, sms); }

nvfp4kv_status launch_matmul(const MatmulArgs& a, const void* w_codes, const void* x_codes,
                             cudaStream_t stream) {
    if (a.offsets)
        return a.y_f32 ? launch_any<true, true>(a, w_codes, x_codes, stream)
                       : launch_any<true, false>(a, w_codes, x_codes, stream);
    return a.y_f32 ? launch_any<false, true>(a, w_codes, x_codes, stream)
                   : launch_any<false, false>(a, w_codes, x_codes, stream);
}

}  // namespace nvfp4kv
