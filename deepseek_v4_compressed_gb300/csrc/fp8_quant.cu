// fp8_quant.cu -- E4M3 quantisation of a matrix with one fp32 scale per block
// of 1 x 128 (activations) or 128 x 128 (weights): scale = amax / 448, codes
// = E4M3(x / scale), the rule of the attention output's quantisation (section
// 6.4 of "From MLA to CSA + HCA" places it ahead of the FP8 projection).
//
// One pass: a block's values stay in registers between its maximum and its
// codes.  Bound by HBM: the input read once, one byte and 4/128 bytes written
// per element.  Threads move 16 bytes of input at a time where the alignment
// allows (else single elements).
#include <limits.h>

#include <type_traits>

#include <cuda_fp16.h>

#include "dsv4_common.cuh"
#include "fp8_block.cuh"
#include "host_once.h"
#include "tmap.h"

namespace dsv4 {

struct QuantParams {
    const void* in;
    long long in_stride;
    uint8_t* codes;
    long long codes_stride;
    float* scales;
    long long scales_stride;
    int rows, cols;
    int per_row;                     // blocks in a row
    // the turns of the many-block kernel: blocks side by side (a power of two),
    // turns that cover a row, and from a CTA's turn to its next one
    int wide, wide_shift, col_turns, turn_rows, turn_blocks;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }

template <typename T>
constexpr int kPer = 16 / sizeof(T);                 // elements of a 16-byte chunk
template <typename T>
constexpr int kLanes = 128 / kPer<T>;                // lanes that hold a row of a block: 16 or 32

// A lane's kPer elements of the block that starts at column c0, as fp32, zero
// where the row has ended: side by side (VEC), or kLanes apart, so that what the
// lanes move at a time is side by side (8192 x 8191 bf16: 61.6 us, 77.6 with a
// lane's elements side by side).
template <typename T, bool VEC>
__device__ __forceinline__ void load_chunk(const T* row, int c0, int lane, int cols, float (&x)[kPer<T>])
{
    const int c = VEC ? c0 + lane * kPer<T> : c0 + lane;
    constexpr int step = VEC ? 1 : kLanes<T>;
    if (VEC && kPer<T> <= cols - c) {           // (no sum: cols may be near 2^31)
        const uint4 raw = *reinterpret_cast<const uint4*>(row + c);
        const T* v = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int i = 0; i < kPer<T>; ++i) x[i] = to_f32(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer<T>; ++i) x[i] = i * step < cols - c ? to_f32(row[c + i * step]) : 0.0f;
    }
}

template <int N>
__device__ __forceinline__ float chunk_amax(const float (&x)[N])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}

template <bool VEC, int N>                       // N: 8 of 16-bit elements, 4 of fp32
__device__ __forceinline__ void store_chunk(uint8_t* row, int c0, int lane, int cols, const BlockDiv& div,
                                            const float (&x)[N])
{
    const int c = VEC ? c0 + lane * N : c0 + lane;
    constexpr int step = VEC ? 1 : 128 / N;
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = div.codes<N == 8 ? 1 : 2>(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    if (VEC && N <= cols - c) {
        if constexpr (N == 8) *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(row + c) = w[0];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * step < cols - c) row[c + i * step] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
    }
}

// ---- whole 16-byte chunks, kept as they were read ------------------------------
// Largest magnitude of a chunk; NaN is left out (a chunk of nothing else gives
// NaN, which the maxima over the lanes leave out in turn).
template <typename T>
__device__ __forceinline__ float raw_amax(const uint4& v)
{
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(fabsf(__uint_as_float(v.x)), fabsf(__uint_as_float(v.y))),
                     fmaxf(fabsf(__uint_as_float(v.z)), fabsf(__uint_as_float(v.w))));
    } else {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        auto abs2 = [](uint32_t w) {
            w &= 0x7fff7fffu;
            return *reinterpret_cast<const T2*>(&w);
        };
        const T2 m = __hmax2(__hmax2(abs2(v.x), abs2(v.y)), __hmax2(abs2(v.z), abs2(v.w)));
        return fmaxf(to_f32(m.x), to_f32(m.y));
    }
}

// The two values of a word of 16-bit elements as an fp32 pair.
template <typename T>
__device__ __forceinline__ uint64_t raw_pair(uint32_t w)
{
    if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        return pack2(f.x, f.y);
    } else {
        const float2 f = bf16x2_to_f32x2(w);
        return pack2(f.x, f.y);
    }
}

// Codes by division, for a scale that residual steps do not serve.  Such blocks
// are read a second time, which keeps this out of the common case's registers.
template <typename T>
__device__ __forceinline__ uint2 raw_codes_divided(const uint4& v, float s)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w}, c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            c[0] |= (f32x2_to_e4m3x2(__fdiv_rn(__uint_as_float(w[i]), s), 0.0f) & 0xffu) << (8 * i);
        } else {
            const float2 f = unpack2(raw_pair<T>(w[i]));
            const uint32_t two = f32x2_to_e4m3x2(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s));
            c[i / 2] |= two << (16 * (i % 2));
        }
    }
    return make_uint2(c[0], c[1]);
}

// Codes of a chunk by residual steps: 8 of 16-bit elements, 4 (in x) of fp32.
template <typename T>
__device__ __forceinline__ uint2 raw_codes(const uint4& v, const BlockDiv& div)
{
    if constexpr (sizeof(T) == 4) {
        const uint32_t lo = __byte_perm(v.x, v.y, 0x0073), hi = __byte_perm(v.z, v.w, 0x0073);
        return make_uint2(div.two(pack2(__uint_as_float(v.x), __uint_as_float(v.y))) |
                              (div.two(pack2(__uint_as_float(v.z), __uint_as_float(v.w))) << 16) |
                              (__byte_perm(lo, hi, 0x5410) & 0x80808080u),
                          0);
    } else {
        // the sign bytes are the high bytes of the elements
        const uint32_t lo = div.two<1>(raw_pair<T>(v.x)) | (div.two<1>(raw_pair<T>(v.y)) << 16) |
                            (__byte_perm(v.x, v.y, 0x7531) & 0x80808080u);
        const uint32_t hi = div.two<1>(raw_pair<T>(v.z)) | (div.two<1>(raw_pair<T>(v.w)) << 16) |
                            (__byte_perm(v.z, v.w, 0x7531) & 0x80808080u);
        return make_uint2(lo, hi);
    }
}

template <typename T>
__device__ __forceinline__ void raw_store(uint8_t* at, const uint2& c)
{
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(at) = c.x;
    else *reinterpret_cast<uint2*>(at) = c;
}

// Many 1 x 128 blocks of whole chunks: kLanes lanes a block, four blocks a
// thread and turn, the next turn's loads in flight meanwhile.  A turn of the CTA
// is `wide` blocks (a power of two) of 4 * kGroups / wide rows, a thread's four
// blocks one below the other: they differ by a fixed number of rows, and what a
// turn adds to their addresses is the same for all threads.  The grid stays on
// the machine: a CTA per turn waited at its end for its stores to be
// acknowledged (the fence) with nothing in flight.  HBM bounds it: 8192 x 8192 bf16
// in 32.3 us, 6.3 TB/s.
template <typename T>
__global__ void __launch_bounds__(256, 4) fp8_quant_rows4_kernel(QuantParams Q)
{
    constexpr int kGroups = 256 / kLanes<T>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x % kLanes<T>, group = threadIdx.x / kLanes<T>;
    const int my_block = group & (Q.wide - 1), my_row = group >> Q.wide_shift, step = kGroups >> Q.wide_shift;
    const int my_col = my_block * 128 + lane * kPer<T>;
    const T* in = static_cast<const T*>(Q.in) + my_row * Q.in_stride + my_col;
    uint8_t* codes = Q.codes + my_row * Q.codes_stride + my_col;
    float* scales = Q.scales + my_row * Q.scales_stride + my_block;
    const long long in_step = step * Q.in_stride, codes_step = step * Q.codes_stride, scales_step = step * Q.scales_stride;
    // the turn's place: its first row and block
    const unsigned end = Q.rows;
    unsigned row = blockIdx.x / Q.col_turns * (4 * step);
    int blk = blockIdx.x % Q.col_turns * Q.wide;
    uint4 next[4];
    auto load = [&]() {
        const T* at = in + row * Q.in_stride + blk * 128;
        // rows from the first block's on
        const int rows = blk * 128 + my_col < Q.cols ? static_cast<int>(end - row) - my_row : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            next[u] = make_uint4(0, 0, 0, 0);
            if (u * step < rows) next[u] = *reinterpret_cast<const uint4*>(at + u * in_step);
        }
    };
    load();
    while (row < end) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = next[u];
        const unsigned row0 = row;
        const int blk0 = blk;
        blk += Q.turn_blocks;
        row += Q.turn_rows;
        if (blk >= Q.col_turns * Q.wide) {
            blk -= Q.col_turns * Q.wide;
            row += 4 * step;
        }
        if (row < end) load();
        // the maxima of four blocks over their lanes, each lane ending up with
        // block 2 * (lane / 8 % 2) + lane / 4 % 2 (5 shuffles instead of 16); it
        // forms that block's scale and reciprocal for all
        const bool b1 = lane & 8, b0 = lane & 4;
        float m[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) m[u] = raw_amax<T>(v[u]);
        const float k0 = fmaxf(b1 ? m[2] : m[0], __shfl_xor_sync(0xffffffffu, b1 ? m[0] : m[2], 8));
        const float k1 = fmaxf(b1 ? m[3] : m[1], __shfl_xor_sync(0xffffffffu, b1 ? m[1] : m[3], 8));
        float amax = fmaxf(b0 ? k1 : k0, __shfl_xor_sync(0xffffffffu, b0 ? k0 : k1, 4));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        if (kLanes<T> == 32) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
        const BlockDiv mine(block_scale(amax));
        const int rows = blk0 < Q.per_row - my_block ? static_cast<int>(end - row0) - my_row : 0;
        const bool has = blk0 * 128 + my_col < Q.cols;
        uint8_t* to = codes + row0 * Q.codes_stride + blk0 * 128;
        float* scale_to = scales + row0 * Q.scales_stride + blk0;
        if (__all_sync(0xffffffffu, mine.steps())) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int from = 8 * (u >> 1) + 4 * (u & 1);
                const BlockDiv div(__shfl_sync(0xffffffffu, mine.s, from, kLanes<T>),
                                   __shfl_sync(0xffffffffu, mine.r, from, kLanes<T>));
                const uint2 c = raw_codes<T>(v[u], div);
                if (u * step < rows) {
                    if (has) raw_store<T>(to + u * codes_step, c);
                    if (lane == 0) scale_to[u * scales_step] = div.s;
                }
            }
        } else {
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                const float scale = __shfl_sync(0xffffffffu, mine.s, 8 * (u >> 1) + 4 * (u & 1), kLanes<T>);
                if (u * step < rows) {
                    if (has) {
                        const uint4 w = *reinterpret_cast<const uint4*>(in + row0 * Q.in_stride + blk0 * 128 + u * in_step);
                        raw_store<T>(to + u * codes_step, raw_codes_divided<T>(w, scale));
                    }
                    if (lane == 0) scale_to[u * scales_step] = scale;
                }
            }
        }
    }
    // the kernels behind this one may read the codes before their own wait
    __threadfence();
}

// 1 x 128 blocks, kLanes lanes each, any alignment; a block's values as fp32 in
// registers.  Few blocks are bound by latency: 32 x 8192 bf16 1.9 us, an empty
// launch's time.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(QuantParams Q)
{
    constexpr unsigned kStep = 256 / kLanes<T>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x % kLanes<T>;
    const unsigned blocks = static_cast<unsigned>(Q.per_row) * Q.rows;
    for (unsigned turn = blockIdx.x * kStep; turn < blocks; turn += gridDim.x * kStep) {
        const unsigned at = turn + threadIdx.x / kLanes<T>;
        const int row = at / Q.per_row, kb = at % Q.per_row;
        float x[kPer<T>];
        if (at < blocks) {
            load_chunk<T, VEC>(static_cast<const T*>(Q.in) + row * Q.in_stride, kb * 128, lane, Q.cols, x);
        } else {
#pragma unroll
            for (int i = 0; i < kPer<T>; ++i) x[i] = 0.0f;
        }
        float amax = chunk_amax(x);
#pragma unroll
        for (int o = kLanes<T> / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (at < blocks) {
            const BlockDiv div(block_scale(amax));
            store_chunk<VEC>(Q.codes + row * Q.codes_stride, kb * 128, lane, Q.cols, div, x);
            if (lane == 0) Q.scales[row * Q.scales_stride + kb] = div.s;
        }
    }
    __threadfence();
}

// 128 x 128 blocks in turn, any alignment, the block as fp32 in registers (64
// values a thread).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) fp8_quant_tiles_kernel(QuantParams Q)
{
    constexpr int kRows = 256 / kLanes<T>;               // rows of one pass of the CTA
    constexpr int kPasses = 128 / kRows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float red[2][8];
    const unsigned tiles = static_cast<unsigned>(Q.per_row) * ((Q.rows - 1) / 128 + 1);
    int par = 0;                                         // warps' maxima of every other turn
    for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x, par ^= 1) {
        const int rb = tile / Q.per_row, kb = tile % Q.per_row;
        const int lane = threadIdx.x % kLanes<T>, r0 = rb * 128 + threadIdx.x / kLanes<T>;
        float x[kPasses][kPer<T>];
        float amax = 0.0f;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            if (r0 + p * kRows < Q.rows) {
                load_chunk<T, VEC>(static_cast<const T*>(Q.in) + (r0 + p * kRows) * Q.in_stride, kb * 128, lane, Q.cols,
                                   x[p]);
            } else {
#pragma unroll
                for (int i = 0; i < kPer<T>; ++i) x[p][i] = 0.0f;
            }
        }
#pragma unroll
        for (int p = 0; p < kPasses; ++p) amax = fmaxf(amax, chunk_amax(x[p]));
        amax = warp_max(amax);
        if ((threadIdx.x & 31) == 0) red[par][threadIdx.x >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) amax = fmaxf(amax, red[par][w]);
        const BlockDiv div(block_scale(amax));
#pragma unroll
        for (int p = 0; p < kPasses; ++p)
            if (r0 + p * kRows < Q.rows)
                store_chunk<VEC>(Q.codes + (r0 + p * kRows) * Q.codes_stride, kb * 128, lane, Q.cols, div, x[p]);
        if (threadIdx.x == 0) Q.scales[rb * Q.scales_stride + kb] = div.s;
    }
    __threadfence();
}

// The same for whole chunks, kept as they were read (32 or 64 registers): three
// CTAs an SM, one loading while others work.  8192 x 8192 bf16 33.6 us, 6.0 TB/s.
template <typename T>
__global__ void __launch_bounds__(256, 3) fp8_quant_tiles_raw_kernel(QuantParams Q)
{
    constexpr int kRows = 256 / kLanes<T>;
    constexpr int kPasses = 128 / kRows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float red[2][8];
    const unsigned tiles = static_cast<unsigned>(Q.per_row) * ((Q.rows - 1) / 128 + 1);
    int par = 0;
    for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x, par ^= 1) {
        const int rb = tile / Q.per_row, kb = tile % Q.per_row;
        const int c = kb * 128 + (threadIdx.x % kLanes<T>) * kPer<T>, r0 = rb * 128 + threadIdx.x / kLanes<T>;
        const int rows = c < Q.cols ? Q.rows - r0 : 0;          // of this thread's column
        const T* in = static_cast<const T*>(Q.in) + r0 * Q.in_stride + c;
        uint4 v[kPasses];
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            v[p] = make_uint4(0, 0, 0, 0);
            if (p * kRows < rows) v[p] = *reinterpret_cast<const uint4*>(in + p * kRows * Q.in_stride);
        }
        float amax = 0.0f;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) amax = fmaxf(amax, raw_amax<T>(v[p]));
        amax = warp_max(amax);
        if ((threadIdx.x & 31) == 0) red[par][threadIdx.x >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) amax = fmaxf(amax, red[par][w]);
        const BlockDiv div(block_scale(amax));
        uint8_t* out = Q.codes + r0 * Q.codes_stride + c;
        if (div.steps()) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
                if (p * kRows < rows) raw_store<T>(out + p * kRows * Q.codes_stride, raw_codes<T>(v[p], div));
        } else {
#pragma unroll 1
            for (int p = 0; p < kPasses; ++p)
                if (p * kRows < rows)
                    raw_store<T>(out + p * kRows * Q.codes_stride,
                                 raw_codes_divided<T>(*reinterpret_cast<const uint4*>(in + p * kRows * Q.in_stride), div.s));
        }
        if (threadIdx.x == 0) Q.scales[rb * Q.scales_stride + kb] = div.s;
    }
    __threadfence();
}

// The same for many blocks of fp32: one CTA an SM, kRing bytes of blocks on their
// way into shared memory while it works on one.  A thread copies what it reads
// itself later, so that only the maximum is exchanged.  HBM bounds it: 8192 x 8192
// in 53.5 us, 6.3 TB/s, against 58.0 us with blocks in registers.  16-bit blocks
// are half as large and gain nothing by it (33.6 us in registers, 39.9 us here).
constexpr int kRing = 3 * 65536, kRingThreads = 512;

template <typename T>
__global__ void __launch_bounds__(kRingThreads, 1) fp8_quant_tiles_ring_kernel(QuantParams Q)
{
    constexpr int kRows = kRingThreads / kLanes<T>;
    constexpr int kPasses = 128 / kRows;
    constexpr int kSlots = kRing / (128 * 128 * static_cast<int>(sizeof(T)));
    constexpr int kWarps = kRingThreads / 32;
    extern __shared__ uint4 ring[];                      // [slot][pass][thread]
    __shared__ float red[2][kWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const unsigned tiles = static_cast<unsigned>(Q.per_row) * ((Q.rows - 1) / 128 + 1);
    const int lane_col = (threadIdx.x % kLanes<T>) * kPer<T>, lane_row = threadIdx.x / kLanes<T>;
    const T* const base = static_cast<const T*>(Q.in);
    uint4* const mine = ring + threadIdx.x;
    auto fetch = [&](unsigned tile, int slot) {
        if (tile < tiles) {
            const int c = tile % Q.per_row * 128 + lane_col, r0 = tile / Q.per_row * 128 + lane_row;
            const int rows = c < Q.cols ? Q.rows - r0 : 0;
            const T* in = base + r0 * Q.in_stride + c;
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                const bool has = p * kRows < rows;
                // no bytes are read where there are none, zeros are written
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 static_cast<uint32_t>(__cvta_generic_to_shared(mine + (slot * kPasses + p) * kRingThreads))),
                             "l"(has ? in + p * kRows * Q.in_stride : base), "r"(has ? 16 : 0)
                             : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kSlots; ++s) fetch(blockIdx.x + s * gridDim.x, s);
    int par = 0, slot = 0;
    for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x, par ^= 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
        uint4 v[kPasses];
#pragma unroll
        for (int p = 0; p < kPasses; ++p) v[p] = mine[(slot * kPasses + p) * kRingThreads];
        float amax = 0.0f;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) amax = fmaxf(amax, raw_amax<T>(v[p]));
        amax = warp_max(amax);
        if ((threadIdx.x & 31) == 0) red[par][threadIdx.x >> 5] = amax;
        __syncthreads();
        // the slot has been read
        fetch(tile + kSlots * gridDim.x, slot);
        slot = slot + 1 == kSlots ? 0 : slot + 1;
        amax = red[par][threadIdx.x % kWarps];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const BlockDiv div(block_scale(amax));
        const int rb = tile / Q.per_row, kb = tile % Q.per_row;
        const int c = kb * 128 + lane_col, r0 = rb * 128 + lane_row;
        const int rows = c < Q.cols ? Q.rows - r0 : 0;
        uint8_t* out = Q.codes + r0 * Q.codes_stride + c;
        if (div.steps()) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
                if (p * kRows < rows) raw_store<T>(out + p * kRows * Q.codes_stride, raw_codes<T>(v[p], div));
        } else {
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
                if (p * kRows < rows) raw_store<T>(out + p * kRows * Q.codes_stride, raw_codes_divided<T>(v[p], div.s));
        }
        if (threadIdx.x == 0) Q.scales[rb * Q.scales_stride + kb] = div.s;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __threadfence();
}

template <typename T, bool VEC>
static cudaError_t launch_quant(QuantParams& Q, int block_rows, cudaStream_t stream)
{
    const unsigned blocks = static_cast<unsigned>(Q.per_row) * Q.rows;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (block_rows == 1) {
        constexpr unsigned step = 256 / kLanes<T>;
        const unsigned sms = sm_count();
        // four blocks a thread once that occupies half of the CTAs: rows of 8192
        // bf16, us by this kernel and the other: 256 3.83, 3.43; 512 4.65, 5.21;
        // 1024 6.73, 8.50
        if (VEC && Q.cols % kPer<T> == 0 && blocks >= 4u * step * 2u * sms) {
            // as many blocks side by side as divide a row: a row of 7 as 8 side by
            // side took 40.4 us for 134 MB of bf16, one by one it takes 31.9
            Q.wide_shift = sizeof(T) == 4 ? 3 : 4;
            while (Q.per_row & ((1 << Q.wide_shift) - 1)) --Q.wide_shift;
            const unsigned turn = 4 * (step >> Q.wide_shift), row_turns = (Q.rows - 1u) / turn + 1;
            // few rows leave too much of their turns empty
            if (static_cast<unsigned long long>(row_turns) * turn * 4 <= Q.rows * 5ull) {
                const int grid = 4 * sms;
                Q.wide = 1 << Q.wide_shift;
                Q.col_turns = Q.per_row / Q.wide;
                Q.turn_rows = grid / Q.col_turns * turn;
                Q.turn_blocks = grid % Q.col_turns * Q.wide;
                cfg.gridDim = dim3(grid, 1, 1);
                return cudaLaunchKernelEx(&cfg, fp8_quant_rows4_kernel<T>, Q);
            }
        }
        const unsigned ctas = (blocks + step - 1) / step;
        cfg.gridDim = dim3(ctas < 8 * sms ? ctas : 8 * sms, 1, 1);
        return cudaLaunchKernelEx(&cfg, fp8_quant_rows_kernel<T, VEC>, Q);
    }
    const unsigned tiles = Q.per_row * ((Q.rows - 1u) / 128u + 1u), most = 3u * sm_count();
    // 512 x 128 x 128 fp32: 10.9 us by the ring, 11.6 without; 256: 7.2 and 6.8 us
    if (VEC && sizeof(T) == 4 && Q.cols % kPer<T> == 0 && tiles > most) {
        static PerDeviceOnce once;
        if (!once.run([] {
                return cudaFuncSetAttribute(fp8_quant_tiles_ring_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            kRing) == cudaSuccess;
            }))
            return cudaErrorInvalidConfiguration;
        cfg.gridDim = dim3(sm_count(), 1, 1);
        cfg.blockDim = dim3(kRingThreads, 1, 1);
        cfg.dynamicSmemBytes = kRing;
        return cudaLaunchKernelEx(&cfg, fp8_quant_tiles_ring_kernel<float>, Q);
    }
    cfg.gridDim = dim3(tiles < most ? tiles : most, 1, 1);
    if (VEC && Q.cols % kPer<T> == 0) return cudaLaunchKernelEx(&cfg, fp8_quant_tiles_raw_kernel<T>, Q);
    return cudaLaunchKernelEx(&cfg, fp8_quant_tiles_kernel<T, VEC>, Q);
}

template <typename T>
static cudaError_t launch_quant(QuantParams& Q, int block_rows, cudaStream_t stream)
{
    // whole chunks on their own alignment, input and codes
    const uintptr_t per = kPer<T>;
    const bool vec = (reinterpret_cast<uintptr_t>(Q.in) & 15) == 0 && (reinterpret_cast<uintptr_t>(Q.codes) & (per - 1)) == 0 &&
                     (Q.rows == 1 || (Q.in_stride % per == 0 && Q.codes_stride % per == 0));
    return vec ? launch_quant<T, true>(Q, block_rows, stream) : launch_quant<T, false>(Q, block_rows, stream);
}

}  // namespace dsv4

using namespace dsv4;

extern "C" dsv4_status dsv4_fp8_block_quant(const dsv4_fp8_quant_args* a, dsv4_stream_t stream)
{
    if (a == nullptr || a->rows < 0 || a->cols < 0 || a->in_stride < 0 || a->codes_stride < 0 ||
        a->scales_stride < 0)
        return DSV4_ERR_INVALID;
    if (a->in_type < DSV4_BF16 || a->in_type > DSV4_E4M3) return DSV4_ERR_INVALID;
    if (a->in_type == DSV4_E4M3 || (a->block_rows != 1 && a->block_rows != 128)) return DSV4_ERR_UNSUPPORTED;
    if (a->rows == 0 || a->cols == 0) return DSV4_OK;
    if (!a->in_dev || !a->codes_dev || !a->scales_dev) return DSV4_ERR_INVALID;
    const long long per_row = (static_cast<long long>(a->cols) + 127) / 128;
    const long long srows = (static_cast<long long>(a->rows) + a->block_rows - 1) / a->block_rows;
    if (per_row * a->rows > INT_MAX) return DSV4_ERR_UNSUPPORTED;
    const uintptr_t esz = a->in_type == DSV4_FP32 ? 4 : 2;
    if ((a->rows > 1 && (a->in_stride < a->cols || a->codes_stride < a->cols)) ||
        (srows > 1 && a->scales_stride < per_row) || (reinterpret_cast<uintptr_t>(a->in_dev) & (esz - 1)) ||
        (reinterpret_cast<uintptr_t>(a->scales_dev) & 3))
        return DSV4_ERR_SHAPE;
    QuantParams Q;
    Q.in = a->in_dev;
    Q.in_stride = a->in_stride;
    Q.codes = static_cast<uint8_t*>(a->codes_dev);
    Q.codes_stride = a->codes_stride;
    Q.scales = a->scales_dev;
    Q.scales_stride = a->scales_stride;
    Q.rows = a->rows;
    Q.cols = a->cols;
    Q.per_row = static_cast<int>(per_row);
    Q.wide = Q.wide_shift = Q.col_turns = Q.turn_rows = Q.turn_blocks = 0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (a->in_type == DSV4_BF16) e = launch_quant<__nv_bfloat16>(Q, a->block_rows, s);
    else if (a->in_type == DSV4_FP16) e = launch_quant<__half>(Q, a->block_rows, s);
    else e = launch_quant<float>(Q, a->block_rows, s);
    if (e == cudaSuccess) return DSV4_OK;
    (void)cudaGetLastError();
    return DSV4_ERR_CUDA;
}
