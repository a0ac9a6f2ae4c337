// Operators that write the paged latent cache and summarise it: the append of new tokens'
// rows (RMS norm, position rotation, 16-bit or "FP8 with scale" rows) and the 8-bit page keys
// that page selection scores.  Formulas, layouts and errors: include/mla_decode.h.

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "../../include/mla_decode.h"
#include "host_util.cuh"
#include "ptx.cuh"
#include "scheduler.cuh"

namespace mla {

constexpr int kLatent = 512;           // latent columns of a row
constexpr int kRopeCols = 64;          // position columns of a 576-wide row
constexpr int kFp8RowBytes = 656;      // 512 e4m3, 4 float32 scales, 64 bfloat16
constexpr int kFp8ScaleOff = 512;
constexpr int kFp8RopeOff = 528;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126: the least scale, so that no block divides by zero

// One 32-bit word of two 16-bit values <-> two floats.
template <bool kFp16>
__device__ __forceinline__ float2 unpack16(uint32_t w)
{
    if constexpr (kFp16) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    } else {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack16(float a, float b)
{
    if constexpr (kFp16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

template <bool kFp16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16<kFp16>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <bool kFp16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack16<kFp16>(x[0], x[1]), pack16<kFp16>(x[2], x[3]), pack16<kFp16>(x[4], x[5]),
                      pack16<kFp16>(x[6], x[7]));
}

// ------------------------------------------------------------------ append
struct AppendParams {
    const uint8_t* latent;   // 16-bit rows of 512, latent_stride bytes apart
    const uint8_t* k_pe;     // 16-bit rows of 64 (null: 512-wide rows)
    const uint8_t* weight;   // 16-bit [512] (null: no norm)
    const int32_t* positions;
    const float* cos_sin;    // [max_position, 64]: 32 cosines, 32 sines
    const int32_t* slots;
    uint8_t* cache;
    const uint8_t* q_pe;     // null: no queries
    uint8_t* q;              // row (t, h): position columns at byte 1024
    int* status;
    long long latent_stride, k_pe_stride, q_pe_tok, q_pe_head, q_tok, q_head;  // bytes
    float eps;
    int tokens, h_q, max_position, cache_rows, interleaved, kv_blocks, d_qk;
};

constexpr int kAppendThreads = 128;
constexpr int kAppendTokens = kAppendThreads / 32;  // cache rows per block (one warp each)
constexpr int kAppendHeads = 2;                     // query heads per thread

// The pass is bound by memory (a token of 128 heads moves 32.8 KB of query columns and 2.3 KB of
// row, and computes 8 flops per query value), or, for a decode step, by the latency of one launch:
// so everything is one launch.  Blocks [0, kv_blocks) take the cache rows, one warp per token:
// lane l owns latent columns [16 l, 16 l + 16), the sum of squares and the block maxima (128
// columns = 8 lanes) go through shuffles, and a row leaves in one pass.  The other blocks rotate
// the queries: four threads per (token, head), each with 16 of the 64 columns as two 16-byte
// loads, and two heads per thread, which share the 64 bytes of cosines and sines.  A thread loads
// all that it needs before it stores, so q_pe may be the columns of q themselves.
template <bool kFp16, bool kFp8>
__global__ void __launch_bounds__(kAppendThreads) mla_append_kernel(const AppendParams p)
{
    const int lane = threadIdx.x & 31;
    if (static_cast<int>(blockIdx.x) < p.kv_blocks) {
        const int t = blockIdx.x * kAppendTokens + (threadIdx.x >> 5);
        if (t >= p.tokens) return;
        const int slot = p.slots[t];
        const uint4* src = reinterpret_cast<const uint4*>(p.latent + t * p.latent_stride) + 2 * lane;
        const uint4 raw0 = src[0], raw1 = src[1];
        int pos = 0;
        float cs = 1.f, sn = 0.f, a = 0.f, b = 0.f;
        bool pos_ok = true;
        if (p.k_pe) {
            pos = p.positions[t];
            pos_ok = pos >= 0 && pos < p.max_position;
            const uint16_t* k = reinterpret_cast<const uint16_t*>(p.k_pe + t * p.k_pe_stride);
            // pair `lane`: columns (2 l, 2 l + 1), or (l, l + 32)
            const uint32_t w = p.interleaved ? reinterpret_cast<const uint32_t*>(k)[lane]
                                             : (static_cast<uint32_t>(k[lane]) | (static_cast<uint32_t>(k[lane + 32]) << 16));
            const float2 f = unpack16<kFp16>(w);
            a = f.x;
            b = f.y;
            if (pos_ok) {
                cs = __ldg(p.cos_sin + static_cast<size_t>(pos) * kRopeCols + lane);
                sn = __ldg(p.cos_sin + static_cast<size_t>(pos) * kRopeCols + 32 + lane);
            }
        }
        if (slot < 0) return;  // padding: no row
        if (slot >= p.cache_rows || !pos_ok) {
            if (lane == 0 && p.status) atomicCAS(p.status, 0, MLA_ERR_DEVICE_CHECK);
            return;
        }
        float x[16];
        {
            float lo[8], hi[8];
            unpack8<kFp16>(raw0, lo);
            unpack8<kFp16>(raw1, hi);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = lo[i];
                x[8 + i] = hi[i];
            }
        }
        if (p.weight) {  // y = x * rsqrt(mean x^2 + eps) * w, in 32 bits
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            const float r = rsqrtf(s * (1.0f / kLatent) + p.eps);
            const uint4* wv = reinterpret_cast<const uint4*>(p.weight) + 2 * lane;
            float w0[8], w1[8];
            unpack8<kFp16>(__ldg(wv), w0);
            unpack8<kFp16>(__ldg(wv + 1), w1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = x[i] * r * w0[i];
                x[8 + i] = x[8 + i] * r * w1[i];
            }
        }
        const float u = a * cs - b * sn, v = b * cs + a * sn;
        uint8_t* rope;  // the row's 64 position columns
        if constexpr (kFp8) {
            uint8_t* row = p.cache + static_cast<size_t>(slot) * kFp8RowBytes;
            // scale of the 128 columns of these 8 lanes: amax / 448 (as a product), at least 2^-126;
            // the code is the e4m3 value next to y / scale
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
            for (int o = 4; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float scale = fmaxf(m * (1.0f / 448.0f), kTinyScale);
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = 0;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 y2 = make_float2(__fdiv_rn(x[4 * i + 2 * j], scale), __fdiv_rn(x[4 * i + 2 * j + 1], scale));
                    c[i] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y2, __NV_SATFINITE, __NV_E4M3)) << (16 * j);
                }
            }
            reinterpret_cast<uint4*>(row)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
            if ((lane & 7) == 0) reinterpret_cast<float*>(row + kFp8ScaleOff)[lane >> 3] = scale;
            rope = row + kFp8RopeOff;
        } else {
            uint8_t* row = p.cache + static_cast<size_t>(slot) * p.d_qk * 2;
            float lo[8], hi[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo[i] = x[i];
                hi[i] = x[8 + i];
            }
            reinterpret_cast<uint4*>(row)[2 * lane] = pack8<kFp16>(lo);
            reinterpret_cast<uint4*>(row)[2 * lane + 1] = pack8<kFp16>(hi);
            rope = row + kLatent * 2;
        }
        if (p.k_pe) {
            const uint32_t w = pack16<kFp16>(u, v);
            if (p.interleaved) {
                reinterpret_cast<uint32_t*>(rope)[lane] = w;
            } else {
                reinterpret_cast<uint16_t*>(rope)[lane] = static_cast<uint16_t>(w);
                reinterpret_cast<uint16_t*>(rope)[lane + 32] = static_cast<uint16_t>(w >> 16);
            }
        }
        return;
    }
    // ---- queries
    const int per_token = (p.h_q + kAppendHeads - 1) / kAppendHeads * 4;
    const unsigned i = (blockIdx.x - p.kv_blocks) * kAppendThreads + threadIdx.x;
    const int t = static_cast<int>(i / static_cast<unsigned>(per_token));
    if (t >= p.tokens) return;
    const int rest = static_cast<int>(i - static_cast<unsigned>(t) * per_token);
    const int c = rest & 3, h0 = (rest >> 2) * kAppendHeads;
    // bytes of the thread's two 16-byte words in a row: 16 columns in a run, or 8 of each half
    const int at0 = p.interleaved ? 32 * c : 16 * c, at1 = p.interleaved ? 32 * c + 16 : 64 + 16 * c;
    uint4 raw[kAppendHeads][2];
#pragma unroll
    for (int h = 0; h < kAppendHeads; ++h) {
        const uint8_t* src = p.q_pe + t * p.q_pe_tok + (h0 + h < p.h_q ? h0 + h : h0) * p.q_pe_head;
        raw[h][0] = *reinterpret_cast<const uint4*>(src + at0);
        raw[h][1] = *reinterpret_cast<const uint4*>(src + at1);
    }
    const int pos = p.positions[t];
    if (pos < 0 || pos >= p.max_position) {
        if (rest == 0 && p.status) atomicCAS(p.status, 0, MLA_ERR_DEVICE_CHECK);
        return;
    }
    float cs[8], sn[8];
    {
        const float4* tab = reinterpret_cast<const float4*>(p.cos_sin + static_cast<size_t>(pos) * kRopeCols) + 2 * c;
        const float4 c0 = __ldg(tab), c1 = __ldg(tab + 1), s0 = __ldg(tab + 8), s1 = __ldg(tab + 9);
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    }
#pragma unroll
    for (int h = 0; h < kAppendHeads; ++h) {
        if (h0 + h >= p.h_q) break;
        float w0[8], w1[8];
        unpack8<kFp16>(raw[h][0], w0);
        unpack8<kFp16>(raw[h][1], w1);
        float o0[8], o1[8];
        if (p.interleaved) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o0[2 * k] = w0[2 * k] * cs[k] - w0[2 * k + 1] * sn[k];
                o0[2 * k + 1] = w0[2 * k + 1] * cs[k] + w0[2 * k] * sn[k];
                o1[2 * k] = w1[2 * k] * cs[4 + k] - w1[2 * k + 1] * sn[4 + k];
                o1[2 * k + 1] = w1[2 * k + 1] * cs[4 + k] + w1[2 * k] * sn[4 + k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                o0[k] = w0[k] * cs[k] - w1[k] * sn[k];
                o1[k] = w1[k] * cs[k] + w0[k] * sn[k];
            }
        }
        uint8_t* dst = p.q + t * p.q_tok + (h0 + h) * p.q_head + kLatent * 2;
        *reinterpret_cast<uint4*>(dst + at0) = pack8<kFp16>(o0);
        *reinterpret_cast<uint4*>(dst + at1) = pack8<kFp16>(o1);
    }
}

// ------------------------------------------------------------------ page keys
struct SummarizeParams {
    const uint8_t* cache;
    const int32_t* block_table;
    const int32_t* before;   // lengths before the step, and after it
    const int32_t* after;
    int8_t* keys;
    float* scales;
    int* status;
    int batch, max_blocks, num_blocks, d;
};

// Half a page per stage of a ring that one thread keeps full by bulk copies.
constexpr int kSumStageRows = 32;
constexpr int kSumPhases = 4;                            // threads that share a column group: 8 rows of a stage each
constexpr int kSumRows = kSumStageRows / kSumPhases;
constexpr int kSumWorkers = 72 * kSumPhases;             // 72 groups of 8 columns
constexpr int kSumThreads = kSumWorkers + 32;            // and the loader's warp
constexpr int kSumChunk = 512;                           // requests per prefix sum

template <bool kFp8>
struct SumLayout {
    static constexpr int kStageBytes = kSumStageRows * (kFp8 ? kFp8RowBytes : 1152);  // (narrower rows use less of it)
    static constexpr int kStages = kFp8 ? 4 : 2;
    static constexpr int kOffPart = kStages * kStageBytes;                 // [2 phases][4][73] float2
    static constexpr int kOffFirst = kOffPart + 2 * kSumPhases * 4 * 73 * 8;   // [kSumChunk] first page, [kSumChunk + 1] prefix
    static constexpr int kOffBar = kOffFirst + (2 * kSumChunk + 2) * 4;
    static constexpr int kOffPage = kOffBar + 2 * kStages * 8;             // page of each stage
    static constexpr int kBytes = kOffPage + kStages * 4 + 128;
};
static_assert(2 * (SumLayout<false>::kBytes + 1280) <= 233472 && 2 * (SumLayout<true>::kBytes + 1280) <= 233472,
              "two blocks of an SM share 228 KB");
static_assert(kSumWorkers % 32 == 0 && 2 * kSumWorkers >= 576 && kSumRows >= 1, "whole warps, two columns a worker at the end");
static_assert(SumLayout<false>::kStageBytes % 128 == 0 && SumLayout<true>::kStageBytes % 128 == 0 &&
                  SumLayout<false>::kOffBar % 8 == 0 && SumLayout<true>::kOffBar % 8 == 0, "alignment");

// Sums of pairs of columns that keep what each addition rounds away (in 24 bits: the bound is below).
struct Sum2 {
    float2 hi = {0.f, 0.f}, lo = {0.f, 0.f};

    __device__ __forceinline__ void add(float2 x)
    {
        const float2 s = fadd2(hi, x), b = fsub2(s, hi);
        lo = fadd2(lo, fadd2(fsub2(hi, fsub2(s, b)), fsub2(x, b)));  // s + (that) == hi + x exactly
        hi = s;
    }
};

// Key of a page: the mean of its 64 rows, as 8-bit whole numbers and a scale.  Bound by reading
// the page (73.7 KB of 16-bit rows).  The key's rounding should not depend on the order of the sum,
// so each sum is a pair of floats, kept by packed additions (two columns an instruction, seven per
// pair of values, eight for bfloat16).  With u = 2^-24 and S = sum |r| / 64, what the pair loses: a thread's 16 additions
// round their low parts by at most (1 + 2 + ... + 16) u u S, the 4 phases' meeting by (10 + 64 + 20) u u S:
// less than 2^-40 S together, before the one rounding to float32.  bfloat16 rows are divided by 64 before they
// are added (exact: 2^-139 is the least), so that no partial sum passes the largest float; float16 rows
// cannot get there and are divided at the end.
// Two blocks per SM take every gridDim-th of the list of completed pages, which all blocks derive
// alike (prefix sums over requests).  A block's loader thread looks the pages up and keeps a ring of
// half pages full by bulk copies (a page's rows are contiguous); thread (g, phase) adds columns
// [8 g, 8 g + 8) of 8 rows of a stage, and the phases meet in shared memory once per page.  126 MB of
// pages: 33.1 us, 1.7 times their reads at the copy rate (19.2).  The rest is the start (lengths, table and
// first page in turn: a step of 64 pages takes 8.7) and whole pages dealt out to 296 blocks (1712 pages:
// five or six each, so that the blocks end unevenly).  39.5 with one block per SM and twice the ring, whose
// additions and page ends nothing overlaps; 35.6 with quarter pages.
template <bool kFp16, bool kFp8>
__global__ void __launch_bounds__(kSumThreads, 2) mla_summarize_kernel(const SummarizeParams p)
{
    using L = SumLayout<kFp8>;
    // two values of a row, as they are added
    auto term = [](uint32_t w) {
        if constexpr (kFp16)
            return unpack16<true>(w);
        else
            return fmul2(unpack16<false>(w), make_float2(1.0f / kPage, 1.0f / kPage));
    };
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    // partial sums of columns 8 g + 2 k, + 1: part[2 phase][k][g] and what they rounded away: part[2 phase + 1][k][g]
    float2(*part)[4][73] = reinterpret_cast<float2(*)[4][73]>(smem + L::kOffPart);
    int* first = reinterpret_cast<int*>(smem + L::kOffFirst);
    int* offset = first + kSumChunk;
    volatile int* page_of = reinterpret_cast<volatile int*>(smem + L::kOffPage);
    const uint32_t s_base = smem_addr(smem);
    const uint32_t full = s_base + L::kOffBar, empty = full + 8 * L::kStages;
    __shared__ int warp_sum[kSumThreads / 32];
    __shared__ float warp_max[kSumWorkers / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = tid % 72, phase = tid / 72;
    const int stride = kFp8 ? kFp8RowBytes : p.d * 2;
    if (tid == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, kSumWorkers / 32);
        }
        fence_mbar_init();
    }
    uint32_t stage = 0, parity = 0;  // of the loader, or of a worker
    auto advance = [&] {
        if (++stage == L::kStages) {
            stage = 0;
            parity ^= 1u;
        }
    };
    long long base = 0;  // pages of earlier chunks of requests
    bool ok = true;
    for (int b0 = 0; b0 < p.batch; b0 += kSumChunk) {
        // pages [before / 64, after / 64) of each request are complete now and were not before
        const int here = min(kSumChunk, p.batch - b0);
        int total = 0;
        for (int r0 = 0; r0 < here; r0 += kSumThreads) {
            int n = 0;
            const int r = r0 + tid;
            if (r < here) {
                const int lo = max(p.before[b0 + r], 0) / kPage, hi = max(p.after[b0 + r], 0) / kPage;
                if (hi > p.max_blocks && p.status && blockIdx.x == 0) atomicCAS(p.status, 0, MLA_ERR_DEVICE_CHECK);
                n = max(min(hi, p.max_blocks) - lo, 0);
                first[r] = lo;
            }
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) warp_sum[warp] = x;
            __syncthreads();
            int before_me = total;
            for (int w = 0; w < kSumThreads / 32; ++w) {
                if (w < warp) before_me += warp_sum[w];
                total += warp_sum[w];
            }
            if (r < here) offset[r] = before_me + x - n;
            __syncthreads();
        }
        // this block's pages among [base, base + total): i = skip, skip + gridDim, ...
        const int skip = static_cast<int>((static_cast<long long>(blockIdx.x) - base % gridDim.x + gridDim.x) % gridDim.x);
        if (warp == kSumWorkers / 32) {
            if (lane == 0) {
                for (long long i = skip; i < total && ok; i += gridDim.x) {
                    int lo = 0, hi = here - 1;  // the last request with offset <= i
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (offset[mid] <= i)
                            lo = mid;
                        else
                            hi = mid - 1;
                    }
                    const int j = first[lo] + static_cast<int>(i) - offset[lo];
                    int page = p.block_table[static_cast<size_t>(b0 + lo) * p.max_blocks + j];
                    if (page < 0 || page >= p.num_blocks) {
                        if (p.status) atomicCAS(p.status, 0, MLA_ERR_DEVICE_CHECK);
                        page = -1;
                    }
                    for (int r = 0; r < kPage && ok; r += kSumStageRows, advance()) {
                        if (!(ok = mbar_wait_bounded(empty + 8 * stage, parity ^ 1))) break;
                        page_of[stage] = page;
                        if (page < 0) {
                            mbar_arrive(full + 8 * stage);
                        } else {
                            mbar_arrive_expect_tx(full + 8 * stage, kSumStageRows * stride);
                            bulk_load(s_base + stage * L::kStageBytes,
                                      p.cache + (static_cast<size_t>(page) * kPage + r) * stride, kSumStageRows * stride,
                                      full + 8 * stage);
                        }
                    }
                }
            }
            __syncwarp();
        } else {
            for (long long i = skip; i < total; i += gridDim.x) {
                Sum2 acc[4];
                int page = -1;
#pragma unroll 1
                for (int r0 = 0; r0 < kPage; r0 += kSumStageRows, advance()) {
                    ok = ok && mbar_wait_bounded(full + 8 * stage, parity);
                    page = ok ? page_of[stage] : -1;
                    const uint8_t* row = smem + stage * L::kStageBytes + kSumRows * phase * stride;
                    if (page >= 0 && 8 * g < p.d) {
                        if (kFp8 && g < kLatent / 8) {
#pragma unroll
                            for (int r = 0; r < kSumRows; ++r) {
                                const uint2 raw = *reinterpret_cast<const uint2*>(row + r * kFp8RowBytes + 8 * g);
                                const float sc = *reinterpret_cast<const float*>(row + r * kFp8RowBytes + kFp8ScaleOff + 4 * (g / 16));
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint32_t w = k < 2 ? raw.x : raw.y;
                                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                                        static_cast<__nv_fp8x2_storage_t>(w >> (16 * (k & 1))), __NV_E4M3);
                                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                                    acc[k].add(term(pack16<false>(f.x * sc, f.y * sc)));
                                }
                            }
                        } else {
                            // 16-bit columns: a 16-bit row's, or an FP8 row's position columns
                            const uint8_t* col = row + (kFp8 ? kFp8RopeOff + 16 * (g - kLatent / 8) : 16 * g);
#pragma unroll
                            for (int r = 0; r < kSumRows; ++r) {
                                const uint4 raw = *reinterpret_cast<const uint4*>(col + r * stride);
                                const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) acc[k].add(term(w[k]));
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty + 8 * stage);
                }
                if (page >= 0 && 8 * g < p.d)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        part[2 * phase][k][g] = acc[k].hi;
                        part[2 * phase + 1][k][g] = acc[k].lo;
                    }
                named_barrier_sync(1, kSumWorkers);
                // columns 2 tid, 2 tid + 1: the mean, rounded once to 32 bits
                float m0 = 0.f, m1 = 0.f;
                if (2 * tid < p.d) {
                    Sum2 sum;
                    float2 rest = {0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < kSumPhases; ++q) {
                        sum.add(part[2 * q][tid & 3][tid >> 2]);
                        rest = fadd2(rest, part[2 * q + 1][tid & 3][tid >> 2]);
                    }
                    rest = fadd2(rest, sum.lo);
                    constexpr float kLeft = kFp16 ? 1.0f / kPage : 1.0f;  // (exact: no float16 mean is subnormal)
                    m0 = __fmul_rn(__fadd_rn(sum.hi.x, rest.x), kLeft);
                    m1 = __fmul_rn(__fadd_rn(sum.hi.y, rest.y), kLeft);
                }
                float mx = fmaxf(fabsf(m0), fabsf(m1));
#pragma unroll
                for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                if (lane == 0) warp_max[warp] = mx;
                named_barrier_sync(1, kSumWorkers);  // also: part may be written again
#pragma unroll
                for (int w = 0; w < kSumWorkers / 32; ++w) mx = fmaxf(mx, warp_max[w]);
                const float scale = fmaxf(mx * (1.0f / 127.0f), kTinyScale);
                if (2 * tid < p.d && page >= 0) {
                    const int k0 = max(-127, min(127, __float2int_rn(__fdiv_rn(m0, scale))));
                    const int k1 = max(-127, min(127, __float2int_rn(__fdiv_rn(m1, scale))));
                    reinterpret_cast<char2*>(p.keys + static_cast<size_t>(page) * p.d)[tid] =
                        make_char2(static_cast<char>(k0), static_cast<char>(k1));
                    if (tid == 0) p.scales[page] = scale;
                }
            }
        }
        base += total;
        __syncthreads();  // first and offset may be written again
    }
    if (!ok) {  // a copy that never came: say so, and give those in flight time to land
        if (p.status) atomicCAS(p.status, 0, MLA_ERR_TIMEOUT);
        const uint64_t start = global_timer_ns();
        while (global_timer_ns() - start < 50000000ull) {
        }
    }
}

template <bool kFp16, bool kFp8>
static cudaError_t launch_summarize(int grid, cudaStream_t st, const SummarizeParams& prm)
{
    auto kern = mla_summarize_kernel<kFp16, kFp8>;
    constexpr int smem = SumLayout<kFp8>::kBytes;
    static PerDeviceOnce configured;
    const cudaError_t e =
        configured.run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    kern<<<grid, kSumThreads, smem, st>>>(prm);
    return cudaGetLastError();
}

}  // namespace mla

using namespace mla;

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

extern "C" {

mla_status mla_append_kvcache(const void* latent, long long latent_stride, const void* k_pe, long long k_pe_stride,
                              const void* norm_weight, float norm_eps, const int32_t* positions, const float* cos_sin,
                              int max_position, const int32_t* slots, int num_tokens, void* kvcache, int num_blocks,
                              int page_size, int h_kv, int d_qk, int dtype, int interleaved, const void* q_pe,
                              long long q_pe_token_stride, long long q_pe_head_stride, void* q,
                              long long q_token_stride, long long q_head_stride, int h_q, int32_t* device_status,
                              void* stream)
{
    if (num_tokens < 0 || num_blocks <= 0 || h_kv <= 0 || (interleaved != 0 && interleaved != 1)) return MLA_ERR_INVALID_ARG;
    if (dtype != MLA_BF16 && dtype != MLA_FP16 && dtype != MLA_BF16_FP8KV) return MLA_ERR_INVALID_ARG;
    const bool fp8 = dtype == MLA_BF16_FP8KV;
    if (page_size != kPage || h_kv != 1 || (d_qk != 576 && d_qk != 512) || (fp8 && d_qk != 576)) return MLA_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * kPage >= (1ll << 31)) return MLA_ERR_UNSUPPORTED;
    const bool rope = d_qk == 576;
    if ((q_pe != nullptr) != (q != nullptr) || (!rope && (k_pe || q_pe))) return MLA_ERR_INVALID_ARG;
    if (q_pe && h_q <= 0) return MLA_ERR_INVALID_ARG;
    if (num_tokens == 0) return MLA_OK;
    if (!latent || !slots || !kvcache || (rope && (!k_pe || !positions || !cos_sin || max_position <= 0)))
        return MLA_ERR_INVALID_ARG;
    if (!(norm_eps >= 0.f)) return MLA_ERR_INVALID_ARG;
    // 16-byte accesses: bases aligned, strides a multiple of 8 values; no row runs backwards
    if (!aligned16(latent) || !aligned16(kvcache) || !aligned16(k_pe) || !aligned16(norm_weight) || !aligned16(cos_sin) ||
        !aligned16(q_pe) || !aligned16(q))
        return MLA_ERR_INVALID_ARG;
    const long long strides[] = {latent_stride, rope ? k_pe_stride : 0, q_pe ? q_pe_token_stride : 0,
                                 q_pe ? q_pe_head_stride : 0, q ? q_token_stride : 0, q ? q_head_stride : 0};
    for (long long s : strides)
        if (s < 0 || s % 8 || s > (1ll << 40)) return MLA_ERR_INVALID_ARG;
    if (q) {
        // rows of q that overlap would be written twice: heads inside tokens, or tokens inside heads
        const bool heads_inner = (h_q == 1 || q_head_stride >= d_qk) &&
                                 (num_tokens == 1 || q_token_stride >= (h_q - 1) * q_head_stride + d_qk);
        const bool tokens_inner = (num_tokens == 1 || q_token_stride >= d_qk) &&
                                  (h_q == 1 || q_head_stride >= (num_tokens - 1) * q_token_stride + d_qk);
        if (!heads_inner && !tokens_inner) return MLA_ERR_INVALID_ARG;
    }
    AppendParams prm{};
    prm.latent = static_cast<const uint8_t*>(latent);
    prm.latent_stride = 2 * latent_stride;
    prm.k_pe = static_cast<const uint8_t*>(k_pe);
    prm.k_pe_stride = 2 * k_pe_stride;
    prm.weight = static_cast<const uint8_t*>(norm_weight);
    prm.eps = norm_eps;
    prm.positions = positions;
    prm.cos_sin = cos_sin;
    prm.max_position = max_position;
    prm.slots = slots;
    prm.tokens = num_tokens;
    prm.cache = static_cast<uint8_t*>(kvcache);
    prm.cache_rows = num_blocks * kPage;
    prm.d_qk = d_qk;
    prm.interleaved = interleaved;
    prm.q_pe = static_cast<const uint8_t*>(q_pe);
    prm.q_pe_tok = 2 * q_pe_token_stride;
    prm.q_pe_head = 2 * q_pe_head_stride;
    prm.q = static_cast<uint8_t*>(q);
    prm.q_tok = 2 * q_token_stride;
    prm.q_head = 2 * q_head_stride;
    prm.h_q = h_q;
    prm.status = device_status;
    prm.kv_blocks = (num_tokens + kAppendTokens - 1) / kAppendTokens;
    long long blocks = prm.kv_blocks;
    if (q) {
        const long long items = static_cast<long long>(num_tokens) * ((h_q + kAppendHeads - 1) / kAppendHeads * 4ll);
        if (items >= (1ll << 31)) return MLA_ERR_UNSUPPORTED;
        blocks += (items + kAppendThreads - 1) / kAppendThreads;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(blocks));
    if (fp8)
        mla_append_kernel<false, true><<<grid, kAppendThreads, 0, st>>>(prm);
    else if (dtype == MLA_FP16)
        mla_append_kernel<true, false><<<grid, kAppendThreads, 0, st>>>(prm);
    else
        mla_append_kernel<false, false><<<grid, kAppendThreads, 0, st>>>(prm);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status mla_summarize_pages(const void* kvcache, int num_blocks, int page_size, int h_kv, int d_qk, int dtype,
                               const int32_t* block_table, int max_blocks_per_seq, const int32_t* prev_seqlens,
                               const int32_t* cache_seqlens, int batch, int8_t* page_keys, float* page_scales,
                               int32_t* device_status, void* stream)
{
    if (batch < 0 || num_blocks <= 0 || h_kv <= 0 || max_blocks_per_seq <= 0) return MLA_ERR_INVALID_ARG;
    if (dtype != MLA_BF16 && dtype != MLA_FP16 && dtype != MLA_BF16_FP8KV) return MLA_ERR_INVALID_ARG;
    const bool fp8 = dtype == MLA_BF16_FP8KV;
    if (page_size != kPage || h_kv != 1 || (d_qk != 576 && d_qk != 512) || (fp8 && d_qk != 576)) return MLA_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * kPage >= (1ll << 31)) return MLA_ERR_UNSUPPORTED;
    const long long most = static_cast<long long>(batch) * max_blocks_per_seq;  // pages that a step can complete: counted in int32
    // (requests are counted in steps of a chunk)
    if (most >= (1ll << 31) || batch > (1 << 30)) return MLA_ERR_UNSUPPORTED;
    if (batch == 0) return MLA_OK;
    if (!kvcache || !block_table || !prev_seqlens || !cache_seqlens || !page_keys || !page_scales) return MLA_ERR_INVALID_ARG;
    if (!aligned16(kvcache) || !aligned16(page_keys) || (reinterpret_cast<uintptr_t>(page_scales) & 3)) return MLA_ERR_INVALID_ARG;
    int sms = 0;
    if (!sm_count(&sms)) return MLA_ERR_CUDA;
    SummarizeParams prm{};
    prm.cache = static_cast<const uint8_t*>(kvcache);
    prm.block_table = block_table;
    prm.before = prev_seqlens;
    prm.after = cache_seqlens;
    prm.keys = page_keys;
    prm.scales = page_scales;
    prm.status = device_status;
    prm.batch = batch;
    prm.max_blocks = max_blocks_per_seq;
    prm.num_blocks = num_blocks;
    prm.d = d_qk;
    const int grid = most < 2 * sms ? static_cast<int>(most) : 2 * sms;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = fp8 ? launch_summarize<false, true>(grid, st, prm)
                              : (dtype == MLA_FP16 ? launch_summarize<true, false>(grid, st, prm)
                                                   : launch_summarize<false, false>(grid, st, prm));
    return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
