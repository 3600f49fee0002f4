// fp8_matmul.cu -- grouped FP8 matrix product with a scale for each block of
// 128 (the projection that takes the quantised attention output: section 6.4
// of "From MLA to CSA + HCA").
//
//   out[t][g][j] = sum_b xs[t][g][b] ws[g][j / 128][b] sum_{i in b} x w
#include <limits.h>

#include <atomic>

#include <cuda_fp16.h>

#include "dsv4_common.cuh"
#include "fp8_block.cuh"
#include "host_once.h"
#include "tc_common.cuh"
#include "tmap.h"

namespace dsv4 {

struct MatmulParams {
    int T, G, N, K, kblocks;
    const uint8_t* x;
    long long x_ts, x_gs;
    const float* xs;
    long long xs_ts, xs_gs;
    const uint8_t* w;
    long long w_rs, w_gs;
    const float* ws;
    long long ws_rs, ws_gs;
    int out_type;
    void* out;
    long long out_ts, out_gs;
    float* os;
    long long os_ts, os_gs;
    int* status;
};

// ---- helpers ---------------------------------------------------------------
// acc += f * v on both halves.
__device__ __forceinline__ void ffma2(uint64_t& acc, uint64_t f, uint64_t v)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(f), "l"(v));
}

// Consecutive fp32 columns of this thread's TMEM lane from taddr on, landed on
// return (the load and its wait are one statement: no use can move between).
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[64])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
          "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
          "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
          "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
          "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
        : "r"(taddr)
        : "memory");
}

// use(column, values) over N columns of this thread's lane; done() once the last
// columns are in registers.  64 columns a load: two waits per 128-column block
// (four loads of 32, the next in flight during each use, were 10% slower: the
// compiler moved the registers).
template <int N, typename F, typename G>
__device__ __forceinline__ void tmem_sweep(uint32_t taddr, F&& use, G&& done)
{
    constexpr int C = N < 64 ? N : 64;
#pragma unroll
    for (int c = 0; c < N; c += C) {
        float v[C];
        tmem_load(taddr + c, v);
        if (c + C >= N) done();
        use(c, v);
    }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// Wait for one of this CTA's own copies or products in flight, whatever the
// abort word says, for at most kWaitNs.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = tc::global_timer_ns();
    while (!tc::mbar_try_wait(bar, parity))
        if (tc::global_timer_ns() - t0 > tc::kWaitNs) return;
}

// Round and store one output row's 128-column block jb, held by 16 lanes: lane l
// of them has columns 64 i + 4 l .. + 3 in v[i].  Every lane of the warp calls
// (two rows at a time); `on`: the lane's row exists.
template <int OUT>
__device__ __forceinline__ void store_block(const MatmulParams& P, bool on, int t, int g, int jb, int l,
                                            const float4 (&v)[2], bool vec)
{
    const int j0 = jb * kBlk + 4 * l;
    const long long at = t * P.out_ts + g * P.out_gs + j0;
    if constexpr (OUT == DSV4_E4M3) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = P.N - j0 - 64 * i;                     // columns of this part that exist
            if (n > 0) amax = fmaxf(amax, fabsf(v[i].x));
            if (n > 1) amax = fmaxf(amax, fabsf(v[i].y));
            if (n > 2) amax = fmaxf(amax, fabsf(v[i].z));
            if (n > 3) amax = fmaxf(amax, fabsf(v[i].w));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (!on) return;
        const float s = block_scale(amax), f = steps_factor(s);
        const BlockDiv div(f == 0.0f ? 1.0f : s * f);
        uint8_t* out = static_cast<uint8_t*>(P.out) + at;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t c = div.codes_by_steps(v[i].x * f, v[i].y * f, v[i].z * f, v[i].w * f);
            const int n = P.N - j0 - 64 * i;
            if (vec && n >= 4) {
                *reinterpret_cast<uint32_t*>(out + 64 * i) = c;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < n) out[64 * i + k] = static_cast<uint8_t>(c >> (8 * k));
            }
        }
        if (l == 0) P.os[t * P.os_ts + g * P.os_gs + jb] = s;
    } else {
        if (!on) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = P.N - j0 - 64 * i;
            const float x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            if constexpr (OUT == DSV4_FP32) {
                float* out = static_cast<float*>(P.out) + at + 64 * i;
                if (vec && n >= 4) {
                    *reinterpret_cast<float4*>(out) = v[i];
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < n) out[k] = x[k];
                }
            } else {
                uint16_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    h[k] = OUT == DSV4_BF16 ? f32_to_bf16_bits(x[k]) : __half_as_ushort(__float2half_rn(x[k]));
                uint16_t* out = static_cast<uint16_t*>(P.out) + at + 64 * i;
                if (vec && n >= 4) {
                    *reinterpret_cast<uint2*>(out) = make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16),
                                                                h[2] | (static_cast<uint32_t>(h[3]) << 16));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < n) out[k] = h[k];
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Few tokens: the weights are the M operand (128 output columns of one weight
// block row), NT tokens the N operand, so that reading the weights bounds the
// kernel and a small batch wastes no tensor rows it would pay for.
//   D_b[128 columns x NT] = W_b[128 x 128] X_b[NT x 128]^T     (fp32 in TMEM)
//   acc[column][token] += (ws_b xs_b[token]) D_b[column][token]
// A column's weight scale is one number per block row, so the factor of a
// block depends on the token alone: 128 threads, one per column (TMEM lane),
// read it from shared memory and hold the running sums in registers.
//   warps 0-3: sums, then the joined epilogue;  warp 4: TMA;  warp 5: MMA
// The blocks of k are split over a cluster of `split` CTAs when there are fewer
// column tiles than places for CTAs (two an SM).  Each CTA copies its sums of
// the tokens that CTA r finishes (t % split = r) into r's shared memory, one
// bulk copy each; they are added in the order of the ranks.  (Pushed as 4-byte
// remote stores, 64 tokens' sums took 4100 cycles instead of about 1500.)
// 8 x 1024 x 4096, from HBM: 9.4 us at 1 token, 10.6 at 32, where reading 33.5 MB
// alone takes a launch 6.4 to 7.5 us; the rest is set-up ahead of the first load
// and the exchange and output behind the last.
// ---------------------------------------------------------------------------
constexpr int kStThreads = 192;
constexpr int kStMaxStages = 12;
constexpr int kStWBytes = 128 * 128;

struct StreamParams {
    MatmulParams m;
    int split;                // CTAs of a cluster
    int stages;
    int ntiles, ttiles;
    int x_groups, w_groups;   // 0: one matrix shared by all groups
    int vec;                  // outputs aligned for 4 elements at once
};

template <int NT>
struct StreamCfg {
    static constexpr int kAcc = 4;                               // accumulators in flight
    static constexpr int kCols = kAcc * NT;                      // TMEM columns: 64, 128 or 256, two CTAs an SM
    static constexpr int kStage = kStWBytes + NT * 128;
    static constexpr int kFactors = 2 * 4 * NT * 4;              // two groups of four blocks
    static constexpr int kSums = NT * 512;                        // [split][NT / split][128] fp32
    static constexpr int kFixed = kFactors + 512 /* barriers */ + 1024 /* align */;
};

struct StreamBars {
    uint64_t full[kStMaxStages], empty[kStMaxStages];
    uint64_t acc_full[4], acc_empty[4];
    uint64_t done, recv;
    uint32_t tmem;
    int abort_flag;
};

template <int NT, int OUT>
__global__ void __launch_bounds__(kStThreads)
fp8_matmul_stream_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ StreamParams S)
{
    using C = StreamCfg<NT>;
    const MatmulParams& P = S.m;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = tc::align1024_shared(smem_raw);
    // the CTA's own sums take the stages' place once the products are done;
    // those that others copy here have room of their own, by rank
    float* own = reinterpret_cast<float*>(smem);
    float* recv = reinterpret_cast<float*>(smem + S.stages * C::kStage);
    float* factors = reinterpret_cast<float*>(smem + S.stages * C::kStage + (S.split > 1 ? C::kSums : 0));   // [2][4][NT]
    StreamBars* B = reinterpret_cast<StreamBars*>(reinterpret_cast<uint8_t*>(factors) + C::kFactors);
    volatile int* abort_flag = &B->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int split = S.split, stages = S.stages;
    const int rank = blockIdx.x % split;
    int q = blockIdx.x / split;
    const int tt = q % S.ttiles;
    q /= S.ttiles;
    const int nt = q % S.ntiles, g = q / S.ntiles;
    const int t0 = tt * NT, n0 = nt * 128;
    // this CTA's blocks of k
    const int kb0 = static_cast<int>(static_cast<long long>(P.kblocks) * rank / split);
    const int n_my = static_cast<int>(static_cast<long long>(P.kblocks) * (rank + 1) / split) - kb0;

    const int lsplit = __ffs(split) - 1;                             // split is a power of two
    const int tokens = min(NT, P.T - t0);
    const int my_rows = (tokens - rank + split - 1) >> lsplit;       // tokens this CTA finishes: t % split = rank
    // the whole producer warp goes through its loops and one lane issues, as
    // for the products below
    const bool leader = elect_one();
    auto load = [&](int i, int st) {
        const int k = (kb0 + i) * 128;
        const uint32_t bar = tc::smem_u32(&B->full[st]), at = tc::smem_u32(smem + st * C::kStage);
        if (leader) {
            tc::mbar_arrive_expect_tx(bar, C::kStage);
            tc::tma_load_3d(at, &tm_w, bar, k, n0, S.w_groups ? g : 0);
            tc::tma_load_3d(at + kStWBytes, &tm_x, bar, k, t0, S.x_groups ? g : 0);
        }
        __syncwarp();
    };
    // the producer starts on the first loads while the others set up
    const int n_early = min(n_my, stages);
    if (warp == 4) {
        if (leader) {
            tc::prefetch_tensormap(&tm_w);
            tc::prefetch_tensormap(&tm_x);
            *abort_flag = 0;
        }
        if (lane < stages) {
            tc::mbar_init(tc::smem_u32(&B->full[lane]), 1);
            tc::mbar_init(tc::smem_u32(&B->empty[lane]), 1);
        }
        tc::fence_barrier_init();
        __syncwarp();
        // x may come from the kernel before (and the weights too)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int i = 0; i < n_early; ++i) load(i, i);
    } else if (warp == 5) {
        // not before the kernel ahead has ended: its CTAs may have let this one
        // start without having their own tensor memory yet, and this one would
        // hold theirs while it waits for them
        asm volatile("griddepcontrol.wait;" ::: "memory");
        tc::tmem_alloc(tc::smem_u32(&B->tmem), C::kCols);
        tc::tmem_relinquish();
    } else if (threadIdx.x == 0) {
        for (int i = 0; i < C::kAcc; ++i) {
            tc::mbar_init(tc::smem_u32(&B->acc_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&B->acc_empty[i]), 4);
        }
        tc::mbar_init(tc::smem_u32(&B->done), 1);
        tc::mbar_init(tc::smem_u32(&B->recv), 1);
        tc::fence_barrier_init();
        if (split > 1) tc::mbar_arrive_expect_tx(tc::smem_u32(&B->recv), (split - 1) * my_rows * 512);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (split > 1) tc::cluster_arrive_relaxed();                     // this CTA's barriers are ready
    const uint32_t tmem = B->tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    uint64_t acc[NT / 2];                                 // two tokens each
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) acc[i] = 0;

    if (warp == 4) {
        int issued = n_early, st = 0;
        uint32_t ph = 0;
        for (int i = n_early; i < n_my; ++i) {
            const bool go = tc::mbar_wait(tc::smem_u32(&B->empty[st]), ph, abort_flag, P.status);
            if (!__all_sync(0xffffffffu, go)) break;
            load(i, st);
            issued = i + 1;
            if (++st == stages) {
                st = 0;
                ph ^= 1;
            }
        }
        // no copy may be in flight when the CTA's shared memory goes away
        for (int i = max(0, issued - stages); i < issued; ++i)
            drain(tc::smem_u32(&B->full[i % stages]), (i / stages) & 1);
    } else if (warp == 5) {
        // the whole warp goes through the loop, one lane issues: the
        // descriptors stay in uniform registers (a single-lane loop took about
        // 800 cycles a block to issue its four products)
        constexpr uint32_t idesc = tc::idesc(128, NT, tc::kFmtE4M3, tc::kFmtE4M3);
        const uint64_t a0 = tc::desc_kmajor_sw128(tc::smem_u32(smem));
        const uint32_t full0 = tc::smem_u32(&B->full[0]), empty0 = tc::smem_u32(&B->empty[0]);
        const uint32_t acc_full0 = tc::smem_u32(&B->acc_full[0]), acc_empty0 = tc::smem_u32(&B->acc_empty[0]);
        int st = 0, ab = 0;
        uint32_t st_ph = 0, ab_ph = 1;             // a barrier that has seen no phase yet passes parity 1
        for (int i = 0; i < n_my; ++i) {
            const bool go = tc::mbar_wait(full0 + 8 * st, st_ph, abort_flag, P.status) &&
                            tc::mbar_wait(acc_empty0 + 8 * ab, ab_ph, abort_flag, P.status);
            if (!__all_sync(0xffffffffu, go)) break;
            tc::tc_fence_after();
            const uint64_t a = a0 + st * (C::kStage >> 4), b = a + (kStWBytes >> 4);
            if (leader) {
#pragma unroll
                for (int k = 0; k < 4; ++k)                     // K = 32 codes (32 bytes) per instruction
                    tc::mma_f8f6f4(tmem + ab * NT, a + 2 * k, b + 2 * k, idesc, k > 0 ? 1u : 0u);
                tc::mma_commit(acc_full0 + 8 * ab);
                tc::mma_commit(empty0 + 8 * st);
            }
            __syncwarp();
            if (++st == stages) {
                st = 0;
                st_ph ^= 1;
            }
            if (++ab == C::kAcc) {
                ab = 0;
                ab_ph ^= 1;
            }
        }
        // no product may be in flight when the tensor memory goes away
        if (leader) tc::mma_commit(tc::smem_u32(&B->done));
        __syncwarp();
        drain(tc::smem_u32(&B->done), 0);
    } else {
        const int tid = threadIdx.x;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        // thread c < NT fetches token c's scales four blocks ahead and leaves
        // them, times the weight's, for all
        const bool mine = tid < NT;
        const float* xs = P.xs + (t0 + tid) * P.xs_ts + g * P.xs_gs + kb0;
        const float* ws = P.ws + g * P.ws_gs + nt * P.ws_rs + kb0;
        const bool real = mine && t0 + tid < P.T;
        float nx[4], nw[4];
        auto fetch = [&](int i) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                nx[k] = real && i + k < n_my ? xs[i + k] : 0.0f;
                nw[k] = mine && i + k < n_my ? ws[i + k] : 0.0f;
            }
        };
        fetch(0);
        bool go = true;
        for (int i = 0; i < n_my; ++i) {
            if ((i & 3) == 0) {
                if (mine) {
                    float* f = factors + ((i >> 2) & 1) * 4 * NT + tid;
#pragma unroll
                    for (int k = 0; k < 4; ++k) f[k * NT] = nx[k] * nw[k];
                }
                // the four warps always meet here, a warp that gave up too
                asm volatile("bar.sync 1, 128;" ::: "memory");
                fetch(i + 4);
            }
            const int ab = i % C::kAcc;
            if (go) go = tc::mbar_wait(tc::smem_u32(&B->acc_full[ab]), (i / C::kAcc) & 1, abort_flag, P.status);
            go = __all_sync(0xffffffffu, go);
            if (!go) continue;
            tc::tc_fence_after();
            const ulonglong2* f = reinterpret_cast<const ulonglong2*>(factors + (((i >> 2) & 1) * 4 + (i & 3)) * NT);
            tmem_sweep<NT>(lanes + ab * NT, [&](int c, auto& v) {
                constexpr int n = sizeof(v) / sizeof(float);
#pragma unroll
                for (int k = 0; k < n; k += 4) {
                    const ulonglong2 s = f[(c + k) / 4];
                    ffma2(acc[(c + k) / 2], s.x, pack2(v[k], v[k + 1]));
                    ffma2(acc[(c + k) / 2 + 1], s.y, pack2(v[k + 2], v[k + 3]));
                }
            }, [&]() {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&B->acc_empty[ab]));
            });
        }
    }
    // The tensor memory goes back before any wait for another CTA, so that no
    // CTA that holds some waits for one that waits to get some.
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 5) tc::tmem_dealloc(tmem, C::kCols);
    bool failed = *abort_flag != 0;
    if (warp < 4) {
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
            // row of token t: the tokens of one rank together
            const float2 v = unpack2(acc[t / 2]);
            own[((t & (split - 1)) * (NT >> lsplit) + (t >> lsplit)) * 128 + threadIdx.x] = v.x;
            own[(((t + 1) & (split - 1)) * (NT >> lsplit) + ((t + 1) >> lsplit)) * 128 + threadIdx.x] = v.y;
        }
        if (split > 1) tc::fence_proxy_async_smem();
    }
    __syncthreads();
    if (split > 1) {
        tc::cluster_wait_acquire();                                  // the others' barriers are ready
        if (warp == 0 && lane < split && lane != rank) {
            const int rows = (tokens - lane + split - 1) >> lsplit;
            if (rows > 0)
                tc::bulk_s2s(tc::map_to_rank(tc::smem_u32(recv + rank * (NT >> lsplit) * 128), lane),
                             tc::smem_u32(own + lane * (NT >> lsplit) * 128), rows * 512,
                             tc::map_to_rank(tc::smem_u32(&B->recv), lane));
        }
        __syncwarp();
        const bool got = tc::mbar_wait(tc::smem_u32(&B->recv), 0, abort_flag, P.status);
        failed = !__all_sync(0xffffffffu, got) || failed;
        // what the others sent has left their shared memory
        tc::cluster_arrive_relaxed();
    }
    if (!failed) {
        const int l = lane & 15;
        for (int row0 = 2 * warp; row0 < my_rows; row0 += 2 * (kStThreads / 32)) {
            const int row = row0 + (lane >> 4);
            const bool on = row < my_rows;
            float4 sum[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (on) {
                for (int r = 0; r < split; ++r) {
                    const float* at = (r == rank ? own : recv) + (r * (NT >> lsplit) + row) * 128 + 4 * l;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 v = *reinterpret_cast<const float4*>(at + 64 * i);
                        sum[i].x += v.x;
                        sum[i].y += v.y;
                        sum[i].z += v.z;
                        sum[i].w += v.w;
                    }
                }
            }
            store_block<OUT>(P, on, t0 + (row << lsplit) + rank, g, nt, l, sum, S.vec != 0);
        }
    }
    // the kernels behind this one may read the output before their own wait
    __threadfence();
    // the others have received this CTA's sums
    if (split > 1) tc::cluster_wait_acquire();
}

// ---------------------------------------------------------------------------
// Many tokens: bound by the tensor cores.  Pairs of CTAs (cta_group::2) hold a
// tile of 256 tokens x NC columns (256, or 128 when that leaves pairs without a
// tile), tokens as the M operand: each CTA loads its 128 tokens and its half of
// the columns of a block, and keeps 128 x NC sums.
//   D_b[256 x NC] = X_b[256 x 128] W_b[NC x 128]^T               (fp32 in TMEM)
//   acc[token][column] += (xs_b[token] ws_b[column / 128]) D_b[token][column]
// The tensor memory holds 512 / NC products: the tensor cores write one while 8
// warps per CTA add an older one to their sums: warp w owns tokens 32 (w % 4)
// .. + 31 and the columns of half w / 4, a thread one token's NC / 2 columns (one
// weight scale) in registers.  A block takes the tensor cores 2 NC cycles (128 x
// NC x 128 products an SM at 8192 a cycle), the additions NC issue cycles; a
// product is handed back as soon as its last columns are in registers, before
// they are added.  8192 x 4096 x 8192: 186 us on resident inputs, 156 us with
// the additions left out, 148 us for a library product with one scale in all.  In
// calls one behind the other from HBM it takes 201 us: the board's power limit
// holds the clock at 1650 MHz then.
//   warps 0-7: sums and output;  warp 8: TMA;  warp 9: MMA (in rank 0's CTA);
//   warps 10, 11: the factors xs ws of four blocks at a time into shared memory
// 384 threads start with 168 registers each; warps 8-11 hand some of theirs to
// the sums: 256 x 232 + 128 x 40 = 384 x 168, or 256 x 200 + 128 x 104 where a
// thread has 64 sums (40 registers made the other warps spill).
// The grid is persistent: the loads and products of the next tile go on while
// a tile is rounded, staged in shared memory and stored (TMA).
// ---------------------------------------------------------------------------
constexpr int kPrThreads = 384;
constexpr int kPrStages = 5;
constexpr int kPrX = 128 * 128;                          // a CTA's tokens of a block
constexpr int kPrStaging = 4096;                         // 32 rows x 128 bytes, per warp
constexpr int kPrFactors = 2 * 4 * 2 * 128 * 4;          // two groups of four blocks, per half and token
constexpr int kPrMaxima = 2 * 128 * 4;                   // per half and token
constexpr int kPrBand = 8;                               // token tiles that run next to each other

template <int NC>
struct PairCfg {
    static constexpr int kStage = kPrX + NC / 2 * 128;
    static constexpr int kBufs = 512 / NC;               // products in tensor memory
    static constexpr int kSmem = kPrStages * kStage + 8 * kPrStaging + kPrFactors + kPrMaxima + 512 /* barriers */ +
                                 1024 /* align */;
};
static_assert(PairCfg<256>::kSmem <= 232448, "does not fit shared memory");

struct PairParams {
    MatmulParams m;
    int mtiles, ntiles;
    int tiles;                // of all groups
    int x_groups, w_groups;
    int tma_out;              // the output can be stored by TMA
};

struct PairBars {
    uint64_t full[kPrStages], empty[kPrStages];
    uint64_t acc_full[4], acc_empty[4];
    uint64_t fac_full[2], fac_empty[2];
    uint64_t maxima[4];                                    // of 32 tokens
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(PairBars) <= 512, "barrier room");

// This CTA's bytes of a load whose completion counts on the barrier of the
// pair's first CTA (bit 24 of a cluster address is the CTA's place in the pair).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                              int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar & 0xfeffffffu), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ void mma_pair_f8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on the barrier at this address in both CTAs once every product this
// thread issued is done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Arrive on a barrier of the pair's other CTA (or this one).  No data in memory
// passes with it, only the end of this warp's tensor-memory reads, which the
// tcgen05 fence before it orders: a release at cluster scope here would wait
// for every outstanding access of the thread, about 1500 cycles a block.
__device__ __forceinline__ void mbar_arrive_peer(uint32_t addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void pair_tile(const PairParams& S, int tile, int& g, int& mt, int& nt)
{
    const int per = S.mtiles * S.ntiles;
    g = tile / per;
    const int q = tile % per;
    const int band = q / (kPrBand * S.ntiles);
    const int rows = min(kPrBand, S.mtiles - band * kPrBand);
    const int r = q - band * kPrBand * S.ntiles;
    mt = band * kPrBand + r % rows;
    nt = r / rows;
}

template <int OUT, int NC>
__global__ void __launch_bounds__(kPrThreads, 1)
fp8_matmul_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ PairParams S)
{
    using C = PairCfg<NC>;
    const MatmulParams& P = S.m;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = tc::align1024_shared(smem_raw);
    uint8_t* staging = smem + kPrStages * C::kStage;
    float* factors = reinterpret_cast<float*>(staging + 8 * kPrStaging);          // [group % 2][block][half][token]
    float* maxima = factors + kPrFactors / 4;                                     // [half][token]
    PairBars* B = reinterpret_cast<PairBars*>(maxima + kPrMaxima / 4);
    volatile int* abort_flag = &B->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(tc::cluster_ctarank());
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kPrStages; ++i) {
            tc::mbar_init(tc::smem_u32(&B->full[i]), 1);
            tc::mbar_init(tc::smem_u32(&B->empty[i]), 1);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            tc::mbar_init(tc::smem_u32(&B->acc_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&B->acc_empty[i]), 16);     // the warps of both CTAs
        }
        for (int i = 0; i < 4; ++i) tc::mbar_init(tc::smem_u32(&B->maxima[i]), 2);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(tc::smem_u32(&B->fac_full[i]), 2);
            tc::mbar_init(tc::smem_u32(&B->fac_empty[i]), 8);
        }
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    if (warp == 8 && lane == 0) {
        tc::prefetch_tensormap(&tm_x);
        tc::prefetch_tensormap(&tm_w);
        if (S.tma_out) tc::prefetch_tensormap(&tm_out);
    }
    // both CTAs' barriers exist before either is signalled from the other; the
    // loads and factors then start while the tensor memory is being had (512 x 4096
    // x 4096 12.8 us, 13.4 with one meeting behind both)
    __syncwarp();
    if (warp == 0) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else tc::cluster_arrive_relaxed();
    if (warp == 9) {
        // not before the kernel ahead has ended: its CTAs may have let this one
        // start without having their own tensor memory yet
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         tc::smem_u32(&B->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        tc::tc_fence_before();
    }
    tc::cluster_wait_acquire();
    if (warp == 9) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else tc::cluster_arrive_relaxed();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int KB = P.kblocks;

    if (warp >= 8) {
        if constexpr (NC == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp == 8) {
            const bool leader = elect_one();
            const uint32_t full0 = tc::smem_u32(&B->full[0]), empty0 = tc::smem_u32(&B->empty[0]);
            int i = 0, st = 0;                               // blocks loaded so far, of all tiles
            uint32_t ph = 1;                                 // a barrier that has seen no phase yet passes parity 1
            bool go = true;
            for (int tile = pair; go && tile < S.tiles; tile += pairs) {
                int g, mt, nt;
                pair_tile(S, tile, g, mt, nt);
                const int t0 = mt * 256 + rank * 128, n0 = nt * NC + rank * (NC / 2);
                const int gx = S.x_groups ? g : 0, gw = S.w_groups ? g : 0;
                for (int b = 0; b < KB; ++b, ++i) {
                    go = tc::mbar_wait(empty0 + 8 * st, ph, abort_flag, P.status);
                    go = __all_sync(0xffffffffu, go);
                    if (!go) break;
                    const uint32_t bar = full0 + 8 * st, at = tc::smem_u32(smem) + st * C::kStage;
                    if (leader) {
                        // the first CTA's barrier counts the bytes of both
                        if (rank == 0) tc::mbar_arrive_expect_tx(bar, 2 * C::kStage);
                        tma_load_pair(at, &tm_x, bar, b * 128, t0, gx);
                        tma_load_pair(at + kPrX, &tm_w, bar, b * 128, n0, gw);
                    }
                    __syncwarp();
                    if (++st == kPrStages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            // every stage loaded has been read by the products of both CTAs
            // before the shared memory goes away
            for (int k = max(0, i - kPrStages); k < i; ++k)
                drain(tc::smem_u32(&B->empty[k % kPrStages]), (k / kPrStages) & 1);
        } else if (warp == 9 && rank == 0) {
            tc::cluster_wait_acquire();
            tc::tc_fence_after();
            const uint32_t tmem = B->tmem;
            // the whole warp goes through the loop, one lane issues: the
            // descriptors stay in uniform registers (a single-lane loop took
            // 820 cycles a block to issue it)
            constexpr uint32_t idesc = tc::idesc(256, NC, tc::kFmtE4M3, tc::kFmtE4M3);
            const bool leader = elect_one();
            const uint64_t a0 = tc::desc_kmajor_sw128(tc::smem_u32(smem));
            const uint32_t full0 = tc::smem_u32(&B->full[0]), empty0 = tc::smem_u32(&B->empty[0]);
            const uint32_t acc_full0 = tc::smem_u32(&B->acc_full[0]), acc_empty0 = tc::smem_u32(&B->acc_empty[0]);
            int st = 0, ab = 0;
            uint32_t st_ph = 0, ab_ph = 1;         // a barrier that has seen no phase yet passes parity 1
            bool go = true;
            for (int tile = pair; go && tile < S.tiles; tile += pairs) {
                for (int b = 0; b < KB; ++b) {
                    go = tc::mbar_wait(full0 + 8 * st, st_ph, abort_flag, P.status) &&
                         tc::mbar_wait(acc_empty0 + 8 * ab, ab_ph, abort_flag, P.status);
                    go = __all_sync(0xffffffffu, go);
                    if (!go) break;
                    tc::tc_fence_after();
                    const uint64_t a = a0 + st * (C::kStage >> 4), w = a + (kPrX >> 4);
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_pair_f8f6f4(tmem + ab * NC, a + 2 * k, w + 2 * k, idesc, k > 0 ? 1u : 0u);
                        mma_commit_pair(acc_full0 + 8 * ab);
                        mma_commit_pair(empty0 + 8 * st);
                    }
                    __syncwarp();
                    if (++st == kPrStages) {
                        st = 0;
                        st_ph ^= 1;
                    }
                    ab = (ab + 1) & (C::kBufs - 1);
                    ab_ph ^= ab == 0;
                }
            }
        } else if (warp >= 10) {
            const int q = threadIdx.x - 320;                            // tokens q and q + 64
            int grp = 0;
            bool go = true;
            for (int tile = pair; go && tile < S.tiles; tile += pairs) {
                int g, mt, nt;
                pair_tile(S, tile, g, mt, nt);
                const int t = mt * 256 + rank * 128 + q;
                const float* xs = P.xs + t * P.xs_ts + g * P.xs_gs;
                const float* ws = P.ws + g * P.ws_gs + nt * (NC / 128) * P.ws_rs;
                const bool in0 = t < P.T, in1 = t + 64 < P.T, wide = NC == 256 && (2 * nt + 1) * 128 < P.N;
                for (int b = 0; b < KB; b += 4, ++grp) {
                    go = tc::mbar_wait(tc::smem_u32(&B->fac_empty[grp & 1]), ((grp >> 1) & 1) ^ 1, abort_flag, P.status);
                    go = __all_sync(0xffffffffu, go);
                    if (!go) break;
                    float* f = factors + (grp & 1) * (kPrFactors / 8) + q;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (b + k >= KB) break;
                        const float x0 = in0 ? xs[b + k] : 0.0f, x1 = in1 ? xs[64 * P.xs_ts + b + k] : 0.0f;
                        const float w0 = ws[b + k], w1 = wide ? ws[P.ws_rs + b + k] : 0.0f;
                        f[k * 256] = x0 * w0;
                        f[k * 256 + 64] = x1 * w0;
                        if (NC == 256) {
                            f[k * 256 + 128] = x0 * w1;
                            f[k * 256 + 192] = x1 * w1;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(tc::smem_u32(&B->fac_full[grp & 1]));
                }
            }
        }
    } else {
        if constexpr (NC == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        constexpr int esz = OUT == DSV4_FP32 ? 4 : (OUT == DSV4_E4M3 ? 1 : 2);
        constexpr int cols = NC / 2;                                    // of a thread
        constexpr int per = cols * esz < 128 ? cols : 128 / esz;        // columns of a staging row
        constexpr int rb = per * esz;                                   // its bytes: 128 or 64
        const int half = warp >> 2;
        tc::cluster_wait_acquire();
        tc::tc_fence_after();
        const uint32_t lanes = B->tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + cols * half;
        uint8_t* mine = staging + warp * kPrStaging;
        const float* my_factor = factors + (NC == 256 ? half * 128 : 0) + (warp & 3) * 32 + lane;
        const uint32_t acc_full0 = tc::smem_u32(&B->acc_full[0]);
        const uint32_t acc_empty0 = tc::map_to_rank(tc::smem_u32(&B->acc_empty[0]), 0);
        int ab = 0, grp = 0;
        uint32_t ab_ph = 0;
        bool go = true;
        for (int tile = pair; go && tile < S.tiles; tile += pairs) {
            uint64_t acc[cols / 2];                                      // two columns each
#pragma unroll
            for (int c = 0; c < cols / 2; ++c) acc[c] = 0;
            for (int b = 0; b < KB; ++b) {
                if ((b & 3) == 0) {
                    if (b > 0) {
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&B->fac_empty[grp & 1]));
                        ++grp;
                    }
                    go = tc::mbar_wait(tc::smem_u32(&B->fac_full[grp & 1]), (grp >> 1) & 1, abort_flag, P.status);
                }
                const float f = my_factor[(grp & 1) * (kPrFactors / 8) + (b & 3) * 256];
                const uint64_t ff = pack2(f, f);
                go = go && tc::mbar_wait(acc_full0 + 8 * ab, ab_ph, abort_flag, P.status);
                go = __all_sync(0xffffffffu, go);
                if (!go) break;
                tc::tc_fence_after();
                tmem_sweep<cols>(lanes + ab * NC, [&](int c, auto& v) {
#pragma unroll
                    for (int k = 0; k < 64; k += 2) ffma2(acc[(c + k) / 2], ff, pack2(v[k], v[k + 1]));
                }, [&]() {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_peer(acc_empty0 + 8 * ab);
                });
                ab = (ab + 1) & (C::kBufs - 1);
                ab_ph ^= ab == 0;
            }
            if (!go) break;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&B->fac_empty[grp & 1]));
            ++grp;

            // ---- output: 32 tokens x `cols` columns of the warp
            int g, mt, nt;
            pair_tile(S, tile, g, mt, nt);
            const int tw = mt * 256 + rank * 128 + (warp & 3) * 32;      // the warp's first token
            const int j0 = nt * NC + cols * half;
            float s = 1.0f;
            if constexpr (OUT == DSV4_E4M3) {
                float amax = 0.0f;
                if (j0 + cols <= P.N) {
#pragma unroll
                    for (int c = 0; c < cols / 2; ++c) {
                        const float2 v = unpack2(acc[c]);
                        amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < cols / 2; ++c) {
                        const float2 v = unpack2(acc[c]);
                        if (j0 + 2 * c < P.N) amax = fmaxf(amax, fabsf(v.x));
                        if (j0 + 2 * c + 1 < P.N) amax = fmaxf(amax, fabsf(v.y));
                    }
                }
                if constexpr (NC == 128) {
                    // a block's 128 columns are two warps': they meet over the maxima
                    const int at = (warp & 3) * 32 + lane;
                    const uint32_t bar = tc::smem_u32(&B->maxima[warp & 3]);
                    maxima[half * 128 + at] = amax;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bar);
                    go = tc::mbar_wait(bar, 0, abort_flag, P.status);
                    go = __all_sync(0xffffffffu, go);
                    if (!go) break;
                    amax = fmaxf(amax, maxima[(half ^ 1) * 128 + at]);
                    // and once more before either writes the next tile's
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bar);
                    go = tc::mbar_wait(bar, 1, abort_flag, P.status);
                    go = __all_sync(0xffffffffu, go);
                    if (!go) break;
                }
                s = block_scale(amax);
                if (tw + lane < P.T && j0 < P.N && (NC == 256 || half == 0))
                    P.os[(tw + lane) * P.os_ts + g * P.os_gs + j0 / 128] = s;
            }
            if (tw >= P.T || j0 >= P.N) continue;
            // Every scale goes by residual steps: with a division beside them the code
            // of a tile's columns was so long that fetching it took 2 us a tile, and a
            // branch that scales the sums in place cost the additions above 0.15 us a
            // block (the compiler moved their registers).  4096 x 8 x 1024 x 4096 117 ->
            // 102 us.
            const float f = OUT == DSV4_E4M3 ? steps_factor(s) : 1.0f;
            const BlockDiv div(f == 0.0f ? 1.0f : s * f);
            // staging rows of `per` columns: 16-byte chunk k of row r at chunk
            // k ^ (r % 8), as a TMA store with 128-byte swizzle reads them (64-byte
            // rows: chunk k ^ (r / 2 % 4))
#pragma unroll
            for (int c0 = 0; c0 < cols; c0 += per) {
                // the rows' last store has been read out
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int k = 0; k < rb / 16; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = c0 + k * (16 / esz) + i * (4 / esz);           // columns of this word
                        const float2 u = unpack2(acc[c / 2]);
                        if constexpr (OUT == DSV4_FP32) {
                            w[i] = __float_as_uint((c & 1) ? u.y : u.x);
                        } else if constexpr (OUT == DSV4_BF16) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(u.x, u.y);
                            w[i] = *reinterpret_cast<const uint32_t*>(&h);
                        } else if constexpr (OUT == DSV4_FP16) {
                            const __half2 h = __floats2half2_rn(u.x, u.y);
                            w[i] = *reinterpret_cast<const uint32_t*>(&h);
                        } else {
                            const float2 u2 = unpack2(acc[c / 2 + 1]);
                            w[i] = div.codes_by_steps(u.x * f, u.y * f, u2.x * f, u2.y * f);
                        }
                    }
                    const int at = rb == 128 ? k ^ (lane & 7) : k ^ ((lane >> 1) & 3);
                    *reinterpret_cast<uint4*>(mine + lane * rb + (at << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                const int jc = j0 + c0;                                              // the rows' first column
                if (S.tma_out) {
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && jc < P.N) tma_store_3d(&tm_out, tc::smem_u32(mine), jc, tw, g);
                    continue;
                }
                __syncwarp();
                for (int r0 = 0; r0 < 32; r0 += 128 / rb) {
                    // a row's words by 32 lanes, or two rows' by 16 each
                    const int r = rb == 128 ? r0 : r0 + (lane >> 4), word = rb == 128 ? lane : lane & 15;
                    if (tw + r >= P.T) continue;
                    const int chunk = (word >> 2) ^ (rb == 128 ? r & 7 : (r >> 1) & 3);
                    const uint32_t v = *reinterpret_cast<const uint32_t*>(mine + r * rb + (chunk << 4) + (word & 3) * 4);
                    const long long at = (tw + r) * P.out_ts + g * P.out_gs;
                    const int j = jc + word * (4 / esz);
                    if constexpr (esz == 4) {
                        if (j < P.N) static_cast<uint32_t*>(P.out)[at + j] = v;
                    } else if constexpr (esz == 2) {
                        if (j < P.N) static_cast<uint16_t*>(P.out)[at + j] = static_cast<uint16_t>(v);
                        if (j + 1 < P.N) static_cast<uint16_t*>(P.out)[at + j + 1] = static_cast<uint16_t>(v >> 16);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (j + k < P.N) static_cast<uint8_t*>(P.out)[at + j + k] = static_cast<uint8_t>(v >> (8 * k));
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    // the meeting that the warps without use for the tensor memory went past
    if (warp >= 8 && !(warp == 9 && rank == 0)) tc::cluster_wait_acquire();
    // the kernels behind this one may read the output before their own wait
    __threadfence();
    // neither CTA's shared memory or tensor memory goes away before the
    // other's products and arrivals have ended; the fence above covers these (a
    // release here once more, and one ahead of the loads, cost 0.3 to 0.5 us)
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_arrive_relaxed();
    tc::cluster_wait_acquire();
    tc::tc_fence_after();
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(B->tmem) : "memory");
}

// Tensor map of codes [groups][rows][k]: boxes of 128 codes x `box` rows.
static bool codes_map(CUtensorMap* map, const void* base, int k, int rows, long long row_stride, int groups,
                      long long group_stride, int box)
{
    // a stride of a dimension with one entry is never used, but has to be valid
    const uint64_t rs = rows > 1 ? row_stride : k;
    const uint64_t gs = groups > 1 ? group_stride : rs * rows;
    const uint64_t dims[3] = {static_cast<uint64_t>(k), static_cast<uint64_t>(rows), static_cast<uint64_t>(groups)};
    const uint64_t strides[2] = {rs, gs};
    const uint32_t b[3] = {128, static_cast<uint32_t>(box), 1};
    return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, b, CU_TENSOR_MAP_SWIZZLE_128B);
}

static dsv4_status launch_err(cudaError_t e)
{
    if (e == cudaSuccess) return DSV4_OK;
    (void)cudaGetLastError();
    return DSV4_ERR_CUDA;
}

// k = 0: sums of nothing.  16 lanes per output row and 128 columns.
template <int OUT>
__global__ void __launch_bounds__(256) fp8_matmul_empty_kernel(const __grid_constant__ MatmulParams P)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int nb = (P.N + 127) / 128, lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(P.T) * P.G * nb;
    const float4 zero[2] = {};
    for (long long i0 = blockIdx.x * 16ll + (threadIdx.x >> 5) * 2; i0 < rows; i0 += gridDim.x * 16ll) {
        const long long i = i0 + (lane >> 4);
        store_block<OUT>(P, i < rows, static_cast<int>(i / nb / P.G), static_cast<int>(i / nb % P.G),
                    static_cast<int>(i % nb), lane & 15, zero, false);
    }
    __threadfence();
}

// Clusters of 2, 4 or 8 of the few-token kernel's CTAs (two an SM) that the current
// device has room for at once: a cluster stays within a group of SMs, which leaves
// fewer than there are places for CTAs (152, 74 and 36 on this GPU).
static int clusters_at_once(int size)
{
    static std::atomic<int> known[64][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 2 * sm_count() / size;
    std::atomic<int>& n = known[dev][size / 4 + 1];
    if (n.load() > 0) return n.load();
    // of a kernel without tensor memory: for those that use some the query counts one
    // CTA an SM, also where two run (the times of all three few-token kernels jump at
    // 37 clusters of 8 and 75 of 4)
    const auto kernel = fp8_matmul_empty_kernel<DSV4_BF16>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size, 1, 1);
    cfg.blockDim = dim3(kStThreads, 1, 1);
    cfg.dynamicSmemBytes = 108 * 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int most = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 108 * 1024) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&most, kernel, &cfg) != cudaSuccess || most < 1) {
        (void)cudaGetLastError();
        return 2 * sm_count() / size;
    }
    n.store(most);
    return most;
}

// CTAs that share the blocks of k of one tile: twice as many while every tile's
// cluster still has a place at once and every CTA a block.  (With two CTAs an SM
// counted instead, the last of 37 or 38 and 75 or 76 tiles' clusters ran behind the
// others: 32 tokens, k = 4096, 37 tiles 11.4 us, 75 tiles 15.3.)
static int stream_split(long long tiles, int kblocks)
{
    int split = 1;
    while (split < 8 && split * 2 <= kblocks && tiles <= clusters_at_once(split * 2)) split *= 2;
    return split;
}

template <int NT, int OUT>
static dsv4_status launch_stream(const MatmulParams& P, bool x_shared, bool w_shared, bool vec, cudaStream_t stream)
{
    using C = StreamCfg<NT>;
    StreamParams S;
    S.m = P;
    S.ntiles = (P.N + 127) / 128;
    S.ttiles = (P.T + NT - 1) / NT;
    S.x_groups = !x_shared;
    S.w_groups = !w_shared;
    S.vec = vec;
    const long long tiles = static_cast<long long>(S.ntiles) * S.ttiles * P.G;
    S.split = stream_split(tiles, P.kblocks);
    const long long ctas = tiles * S.split;
    if (ctas > INT_MAX) return DSV4_ERR_UNSUPPORTED;
    // two CTAs share an SM's memory, also when one each would do: clusters of 8
    // with an SM to each CTA did not all find a place (14.0 against 7.5 us for
    // 256 and 128 tokens of 512 x 8192)
    const int room = 108 * 1024 - C::kFixed - (S.split > 1 ? C::kSums : 0);
    int stages = room / C::kStage;
    const int need = C::kSums / C::kStage + 1;               // room for the CTA's own sums
    stages = stages > kStMaxStages ? kStMaxStages : stages;
    const int longest = (P.kblocks + S.split - 1) / S.split;
    if (stages > longest) stages = longest;
    S.stages = stages < need ? need : stages;
    CUtensorMap tw, tx;
    if (!codes_map(&tw, P.w, P.K, P.N, P.w_rs, w_shared ? 1 : P.G, P.w_gs, 128) ||
        !codes_map(&tx, P.x, P.K, P.T, P.x_ts, x_shared ? 1 : P.G, P.x_gs, NT))
        return DSV4_ERR_SHAPE;
    static PerDeviceOnce once;
    if (!once.run([] {
            return cudaFuncSetAttribute(fp8_matmul_stream_kernel<NT, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        108 * 1024) == cudaSuccess;
        })) {
        (void)cudaGetLastError();
        return DSV4_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kStThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(S.stages) * C::kStage + (S.split > 1 ? C::kSums : 0) + C::kFixed;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launch_err(cudaLaunchKernelEx(&cfg, fp8_matmul_stream_kernel<NT, OUT>, tw, tx, S));
}

template <int OUT, int NC>
static dsv4_status launch_pair(const MatmulParams& P, bool x_shared, bool w_shared, cudaStream_t stream)
{
    PairParams S;
    S.m = P;
    S.mtiles = (P.T + 255) / 256;
    S.ntiles = (P.N + NC - 1) / NC;
    const long long tiles = static_cast<long long>(S.mtiles) * S.ntiles * P.G;
    if (tiles > INT_MAX / 2) return DSV4_ERR_UNSUPPORTED;
    S.tiles = static_cast<int>(tiles);
    S.x_groups = !x_shared;
    S.w_groups = !w_shared;
    constexpr int esz = OUT == DSV4_FP32 ? 4 : (OUT == DSV4_E4M3 ? 1 : 2);
    S.tma_out = (reinterpret_cast<uintptr_t>(P.out) & 15) == 0 && (P.T == 1 || P.out_ts * esz % 16 == 0) &&
                (P.G == 1 || P.out_gs * esz % 16 == 0);
    CUtensorMap tx, tw, to;
    if (!codes_map(&tx, P.x, P.K, P.T, P.x_ts, x_shared ? 1 : P.G, P.x_gs, 128) ||
        !codes_map(&tw, P.w, P.K, P.N, P.w_rs, w_shared ? 1 : P.G, P.w_gs, NC / 2))
        return DSV4_ERR_SHAPE;
    to = tx;
    if (S.tma_out) {
        const uint64_t row = (static_cast<uint64_t>(P.N) * esz + 15) / 16 * 16;
        const uint64_t dims[3] = {static_cast<uint64_t>(P.N), static_cast<uint64_t>(P.T), static_cast<uint64_t>(P.G)};
        const uint64_t strides[2] = {P.T > 1 ? static_cast<uint64_t>(P.out_ts) * esz : row,
                                     P.G > 1 ? static_cast<uint64_t>(P.out_gs) * esz : row};
        constexpr bool narrow = NC / 2 * esz < 128;                     // staging rows of 64 bytes
        const uint32_t box[3] = {static_cast<uint32_t>(narrow ? NC / 2 : 128 / esz), 32, 1};
        const CUtensorMapDataType type = esz == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32
                                                  : (esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8);
        if (!encode_tmap(&to, type, 3, P.out, dims, strides, box,
                         narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
            S.tma_out = 0;
    }
    static PerDeviceOnce once;
    if (!once.run([] {
            return cudaFuncSetAttribute(fp8_matmul_pair_kernel<OUT, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        PairCfg<NC>::kSmem) == cudaSuccess;
        })) {
        (void)cudaGetLastError();
        return DSV4_ERR_CUDA;
    }
    const int pairs = sm_count() / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (S.tiles < pairs ? S.tiles : pairs), 1, 1);
    cfg.blockDim = dim3(kPrThreads, 1, 1);
    cfg.dynamicSmemBytes = PairCfg<NC>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launch_err(cudaLaunchKernelEx(&cfg, fp8_matmul_pair_kernel<OUT, NC>, tx, tw, to, S));
}

template <int OUT>
static dsv4_status launch_product(const MatmulParams& P, bool x_shared, bool w_shared, bool vec, cudaStream_t stream)
{
    if (P.K == 0) {
        fp8_matmul_empty_kernel<OUT><<<sm_count(), 256, 0, stream>>>(P);
        return launch_err(cudaGetLastError());
    }
    if (P.T <= 16) return launch_stream<16, OUT>(P, x_shared, w_shared, vec, stream);
    if (P.T <= 32) return launch_stream<32, OUT>(P, x_shared, w_shared, vec, stream);
    if (P.T <= 64) return launch_stream<64, OUT>(P, x_shared, w_shared, vec, stream);
    // Above 64 tokens any kernel serves; the one whose estimate is smallest
    // runs.  In microseconds, with KB blocks of k and w waves of tiles (304
    // places for the few-token kernel's CTAs, 76 for pairs):
    //   few-token kernel, 64 tokens a tile  5.7 + 0.47 w KB / split + (w - 1) 3.6
    //   pairs, 256 x 128 tiles              5.2 + 0.25 KB + (w - 1) (0.26 KB + 0.9)
    //   pairs, 256 x 256 tiles              6.1 + 0.365 KB + (w - 1) (0.31 KB + 2.9)
    // (fitted to 90 shapes of 65 to 1500 tokens with bf16 outputs, all three kernels
    // measured: the choice is 0.6% off the best one on average), and for quantised
    // outputs w times 1.3, 0.9 and 0.8 (2048 x 8192 x 1024 29.1 us by the second,
    // 25.6 by the third; bf16 21.8 and 22.5).
    // Measured in this order, 4096 x 8192: 14.0 / 20.8 / 28.1 at 128 tokens, 36.5 /
    // 21.5 / 28.5 at 512, 70.2 / 36.8 / 29.6 at 1024; 512 x 8192: 7.8 / 20.3 /
    // 28.1 at 128, 14.0 / 20.2 / 28.3 at 1024.
    const long long t64 = (P.T + 63) / 64 * ((P.N + 127ll) / 128) * P.G;
    const long long mt = (P.T + 255) / 256;
    const int sms = sm_count(), split = stream_split(t64, P.kblocks);
    const long long w64 = (t64 * split + 2 * sms - 1) / (2 * sms);
    auto waves = [&](int nc) { return static_cast<double>((mt * ((P.N + nc - 1ll) / nc) * P.G + sms / 2 - 1) / (sms / 2)); };
    const double quant = OUT == DSV4_E4M3 ? 1.0 : 0.0, kb = P.kblocks, w128 = waves(128), w256 = waves(256);
    const double few =
        5.7 + 0.47 * static_cast<double>(w64) * ((P.kblocks + split - 1) / split) + (w64 - 1) * 3.6 + quant * 1.3 * w64;
    const double many128 = 5.2 + 0.25 * kb + (w128 - 1) * (0.26 * kb + 0.9) + quant * 0.9 * w128;
    const double many256 = 6.1 + 0.365 * kb + (w256 - 1) * (0.31 * kb + 2.9) + quant * 0.8 * w256;
    if (few <= many128 && few <= many256) return launch_stream<64, OUT>(P, x_shared, w_shared, vec, stream);
    if (many128 < many256) return launch_pair<OUT, 128>(P, x_shared, w_shared, stream);
    return launch_pair<OUT, 256>(P, x_shared, w_shared, stream);
}

}  // namespace dsv4

using namespace dsv4;

extern "C" dsv4_status dsv4_fp8_block_matmul(const dsv4_fp8_matmul_args* a, dsv4_stream_t stream)
{
    if (a == nullptr || a->num_tokens < 0 || a->groups < 0 || a->n < 0 || a->k < 0) return DSV4_ERR_INVALID;
    if (a->x_token_stride < 0 || a->x_group_stride < 0 || a->xs_token_stride < 0 || a->xs_group_stride < 0 ||
        a->w_row_stride < 0 || a->w_group_stride < 0 || a->ws_row_stride < 0 || a->ws_group_stride < 0 ||
        a->out_token_stride < 0 || a->out_group_stride < 0 || a->os_token_stride < 0 || a->os_group_stride < 0)
        return DSV4_ERR_INVALID;
    if (a->out_type < DSV4_BF16 || a->out_type > DSV4_E4M3) return DSV4_ERR_INVALID;
    if (a->k % 16 != 0 || a->groups > 65535 || a->n > (1 << 24) || a->num_tokens > (1 << 24))
        return DSV4_ERR_UNSUPPORTED;
    if (a->num_tokens == 0 || a->groups == 0 || a->n == 0) return DSV4_OK;
    const bool quant = a->out_type == DSV4_E4M3;
    if (!a->out_dev || (quant && !a->out_scales_dev)) return DSV4_ERR_INVALID;
    if (a->k > 0 && (!a->x_dev || !a->xs_dev || !a->w_dev || !a->ws_dev)) return DSV4_ERR_INVALID;
    auto mis = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
    const uintptr_t esz = a->out_type == DSV4_FP32 ? 4 : (quant ? 1 : 2);
    if (mis(a->x_dev, 16) || mis(a->w_dev, 16) || mis(a->xs_dev, 4) || mis(a->ws_dev, 4) || mis(a->out_dev, esz) ||
        mis(a->out_scales_dev, 4) || mis(a->status_dev, 4))
        return DSV4_ERR_SHAPE;
    const long long T = a->num_tokens, G = a->groups, N = a->n, K = a->k;
    if (K > 0 && ((T > 1 && (a->x_token_stride < K || a->x_token_stride % 16 != 0)) ||
        (N > 1 && (a->w_row_stride < K || a->w_row_stride % 16 != 0)) || (G > 1 && a->x_group_stride % 16 != 0) ||
        (G > 1 && a->w_group_stride % 16 != 0)))
        return DSV4_ERR_SHAPE;
    // outputs of two (token, group) pairs must not overlap: tokens outside
    // groups, or groups outside tokens
    auto apart = [&](long long ts, long long gs, long long len) {
        if (T == 1) return G == 1 || gs >= len;
        if (G == 1) return ts >= len;
        return (gs >= len && ts >= (G - 1) * gs + len) || (ts >= len && gs >= (T - 1) * ts + len);
    };
    if (!apart(a->out_token_stride, a->out_group_stride, N) ||
        (quant && !apart(a->os_token_stride, a->os_group_stride, (N + 127) / 128)))
        return DSV4_ERR_SHAPE;
    MatmulParams P;
    P.T = a->num_tokens;
    P.G = a->groups;
    P.N = a->n;
    P.K = a->k;
    P.kblocks = static_cast<int>((K + 127) / 128);       // 64-bit: k may be near 2^31
    P.x = static_cast<const uint8_t*>(a->x_dev);
    P.x_ts = a->x_token_stride;
    P.x_gs = a->x_group_stride;
    P.xs = a->xs_dev;
    P.xs_ts = a->xs_token_stride;
    P.xs_gs = a->xs_group_stride;
    P.w = static_cast<const uint8_t*>(a->w_dev);
    P.w_rs = a->w_row_stride;
    P.w_gs = a->w_group_stride;
    P.ws = a->ws_dev;
    P.ws_rs = a->ws_row_stride;
    P.ws_gs = a->ws_group_stride;
    P.out_type = a->out_type;
    P.out = a->out_dev;
    P.out_ts = a->out_token_stride;
    P.out_gs = a->out_group_stride;
    P.os = a->out_scales_dev;
    P.os_ts = a->os_token_stride;
    P.os_gs = a->os_group_stride;
    P.status = a->status_dev;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const uintptr_t vb = 4 * esz;
    const bool vec = !mis(a->out_dev, vb) && (T == 1 || a->out_token_stride % 4 == 0) &&
                     (G == 1 || a->out_group_stride % 4 == 0);
    const bool x_shared = G == 1 || a->x_group_stride == 0, w_shared = G == 1 || a->w_group_stride == 0;
    switch (P.out_type) {
    case DSV4_BF16: return launch_product<DSV4_BF16>(P, x_shared, w_shared, vec, st);
    case DSV4_FP16: return launch_product<DSV4_FP16>(P, x_shared, w_shared, vec, st);
    case DSV4_FP32: return launch_product<DSV4_FP32>(P, x_shared, w_shared, vec, st);
    default: return launch_product<DSV4_E4M3>(P, x_shared, w_shared, vec, st);
    }
}
