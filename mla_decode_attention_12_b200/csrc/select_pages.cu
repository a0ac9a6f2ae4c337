// Page selection for block-sparse decoding: every query token scores the 8-bit keys of the pages
// that it sees and keeps the best, as a block table of its own that the paged decode reads.
// Formulas, layouts and errors: include/mla_decode.h.

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "../../include/mla_decode.h"
#include "host_util.cuh"
#include "ptx.cuh"
#include "scheduler.cuh"

namespace mla {

constexpr int kScoreThreads = 512;
constexpr int kTile = 128;                          // pages per tile: the rows (M) of one MMA
constexpr int kMaxHeads = 128;                      // query heads: its columns (N), in groups of 32
constexpr int kKeyBoxBytes = kTile * 64;            // 128 rows x 64 bytes, swizzled in 64-byte rows
constexpr float kTinyQ = 1.17549435e-38f;           // 2^-126

struct SelectParams {
    const uint8_t* q;           // [tokens, h_q, d] 16-bit
    const int8_t* keys;         // [num_blocks, d]
    const float* scales;        // [num_blocks]
    const int32_t* block_table;
    const int32_t* seqlens;
    float* scores;              // [tokens, max_blocks]
    int8_t* q8;                 // [tokens, h_q, d] queries in 8 bits, and their scales
    float* q8_scales;           // [tokens, h_q]
    int32_t* out_table;         // [tokens, topn]
    int32_t* out_lens;          // [tokens]
    int* status;
    int tokens, s_q, h_q, max_blocks, num_blocks, topn, first, last, causal;
};

// Cached rows that token t sees, at most what the block table holds.
__device__ __forceinline__ int seen_by(const SelectParams& p, int t, bool* too_long = nullptr)
{
    const int b = t / p.s_q, s = t - b * p.s_q;
    const long long len = p.seqlens[b];
    const long long n = p.causal ? len - p.s_q + 1 + s : len;
    const long long most = static_cast<long long>(p.max_blocks) * kPage;
    if (too_long) *too_long = n > most;
    return static_cast<int>(n < 0 ? 0 : (n > most ? most : n));
}

__device__ __forceinline__ int tiles_of(int n) { return (pages_of(n) + kTile - 1) / kTile; }

// Asynchronous 16-byte copy into shared memory; zeros when `live` is false (nothing is read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// D(tmem) (+)= A(smem desc) * B(smem desc)^T in 8-bit whole numbers, 32-bit accumulators.
__device__ __forceinline__ void mma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// kind::i8: signed 8-bit A and B, 32-bit accumulators, both operands K-major.
__host__ __device__ constexpr uint32_t instr_desc_i8(int M, int N)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// ------------------------------------------------------------------ queries in 8 bits
// One warp per (token, head): s = max|q| / 127, q8 = q / s rounded to float32 and then to the nearest
// whole number.  The product with the reciprocal is within 3 * 2^-24 of the rounded quotient, relative,
// so at most 2.3e-5 off: it rounds to the same number unless it lies that close to the middle
// between two.  Columns where a lane has such a value are divided (half of the largest value is one, 63.5:
// with 8-bit significands most rows have some).
// Rounding by adding 1.5 * 2^23: the low byte of the sum's pattern is the whole number.
// A kernel of its own: the CTAs of the scoring kernel that share a token would otherwise each do this
// again, which took longer than their reads.
constexpr int kQuantThreads = 256;

__device__ __noinline__ int divided(float x, float s) { return __float2int_rn(__fdiv_rn(x, s)); }

template <int kD, bool kFp16>
__global__ void __launch_bounds__(kQuantThreads) mla_quantize_queries_kernel(const SelectParams p)
{
    constexpr int kPer = kD / 64;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5);
    grid_launch_dependents();
    if (row >= static_cast<long long>(p.tokens) * p.h_q) return;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + row * kD * 2);
    float2 f[kPer];  // columns 64 k + 2 lane, + 1
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const uint32_t raw = __ldg(src + 32 * k + lane);
        if constexpr (kFp16)
            f[k] = __half22float2(*reinterpret_cast<const __half2*>(&raw));
        else
            f[k] = make_float2(__uint_as_float(raw << 16), __uint_as_float(raw & 0xffff0000u));
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) m = fmaxf(m, fmaxf(fabsf(f[k].x), fabsf(f[k].y)));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = fmaxf(m * (1.0f / 127.0f), kTinyQ), inv = __frcp_rn(s);
    uint32_t w[kPer];
    uint32_t close = 0;  // pairs of columns with a value near the middle between two whole numbers
    const float2 inv2 = make_float2(inv, inv), magic = make_float2(12582912.f, 12582912.f);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const float2 y = fmul2(f[k], inv2), t = fadd2(y, magic), d = fsub2(y, fsub2(t, magic));
        if (!(fmaxf(fabsf(d.x), fabsf(d.y)) <= 0.49997f)) close |= 1u << k;  // (or NaN)
        w[k] = __byte_perm(__float_as_uint(t.x), __float_as_uint(t.y), 0x0040);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) reinterpret_cast<uint16_t*>(p.q8 + row * kD)[32 * k + lane] = static_cast<uint16_t>(w[k]);
    if (!(s < 1.0e38f)) close = (1u << kPer) - 1u;  // a row with infinities or NaN: the division's answers
    for (uint32_t todo = __reduce_or_sync(0xffffffffu, close); todo; todo &= todo - 1) {
        const int k = __ffs(todo) - 1;
        // (read again: registers cannot be indexed at run time)
        const uint32_t raw = __ldg(src + 32 * k + lane);
        float2 x;
        if constexpr (kFp16)
            x = __half22float2(*reinterpret_cast<const __half2*>(&raw));
        else
            x = make_float2(__uint_as_float(raw << 16), __uint_as_float(raw & 0xffff0000u));
        const int a = max(-127, min(127, divided(x.x, s))), b = max(-127, min(127, divided(x.y, s)));
        reinterpret_cast<uint16_t*>(p.q8 + row * kD)[32 * k + lane] = static_cast<uint16_t>((a & 0xff) | ((b & 0xff) << 8));
    }
    if (lane == 0) p.q8_scales[row] = s;
}

// ------------------------------------------------------------------ scores
template <int kD>
struct ScoreLayout {
    static constexpr int kBoxes = kD / 64;
    static constexpr int kTileBytes = kBoxes * kKeyBoxBytes;  // 73.7 KB at 576
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kTileBytes;                   // two stages
    static constexpr int kOffRed = kOffK + 2 * kTileBytes;     // [2][4][128] floats: column groups' maxima, by stage
    static constexpr int kOffQs = kOffRed + 2 * 4 * kTile * 4; // [2][128] head scales, by token parity
    static constexpr int kOffBar = kOffQs + 2 * kMaxHeads * 4;
    static constexpr int kBytes = kOffBar + 64 + 1024;
};
static_assert(ScoreLayout<576>::kBytes <= 232448, "shared memory plan exceeds 227 KB");
static_assert(ScoreLayout<576>::kTileBytes % 1024 == 0 && ScoreLayout<512>::kTileBytes % 1024 == 0, "operand alignment");

// Scores.  For a token's pages j, score = max over heads h of (s_h * <q8_h, key_j>) times the page's
// scale, q8_h = rint(q_h / s_h) in [-127, 127] with s_h = max|q_h| / 127: the products are whole
// numbers below 2^24, exact in the 8-bit tensor-core products, so the score is the same bits in any
// order of summation, and which pages win does not depend on the kernel.
//
// It has to read the keys (580 bytes per page and request: one 127th of the page itself).  64 contexts of
// 16k to 131k rows: 32.8 us for the whole selection, its reads 7.9 at the copy rate.  What bounds it: the
// quantizing kernel in front (4.6), the first tile (5), then 4 or 5 tiles of 2.9 us whose reads would take about
// one: three barriers of the block a tile and two stages, so that a stage is filled again only after its
// products; and the choice behind (3).  The
// (token, tile of 128 pages) pairs of the call are laid on a line and each of the SMs takes an equal
// run of it, so that lengths balance.  A tile's keys (rows gathered through the block table) come by
// 16-byte asynchronous copies into the swizzled K-major layout of the MMA, two tiles in flight (the
// first while the queries are still being quantized: programmatic launch); the
// MMA has the pages as rows (M = 128) and the heads as columns, so a thread of the epilogue owns a
// page and takes the maximum over heads in its registers: no exchange between lanes.  A warp fetches the
// same 8 rows of every tile (their pages looked up one tile ahead) and finishes those pages' scores.
// 96 registers: the SM keeps room for a block of the quantizing kernel beside it.
// Per tile: wait for its products, refill its stage, wait for the next tile's keys, start the next
// products, and only then take this one's maxima, so that products and copies run meanwhile.
template <int kD, bool kFp16>
__global__ void __maxnreg__(96) mla_score_pages_kernel(const SelectParams p)
{
    using L = ScoreLayout<kD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_base = smem_addr(smem);
    float(*red)[4][kTile] = reinterpret_cast<float(*)[4][kTile]>(smem + L::kOffRed);
    float(*qscale)[kMaxHeads] = reinterpret_cast<float(*)[kMaxHeads]>(smem + L::kOffQs);
    const uint32_t bar = s_base + L::kOffBar;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 16);
    __shared__ int sh_token, sh_tile, warp_tot[kScoreThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_launch_dependents();
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
        sh_token = p.tokens;
        sh_tile = 0;
    }

    // ---- this CTA's run [t_lo, t_hi) of the line of tiles: total first, then the token t_lo falls into
    auto block_scan = [&](int x, int& total) {  // exclusive
        int incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        __syncthreads();
        if (lane == 31) warp_tot[warp] = incl;
        __syncthreads();
        int before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < kScoreThreads / 32; ++w) {
            if (w < warp) before += warp_tot[w];
            total += warp_tot[w];
        }
        return before + incl - x;
    };
    int t_lo = 0, t_hi = 0;
    auto cut = [&](int line) {
        t_lo = static_cast<int>(static_cast<long long>(line) * blockIdx.x / gridDim.x);
        t_hi = static_cast<int>(static_cast<long long>(line) * (blockIdx.x + 1) / gridDim.x);
    };
    auto tiles_at = [&](int t) {
        bool too_long;
        const int n = tiles_of(seen_by(p, t, &too_long));
        if (too_long && blockIdx.x == 0 && p.status) atomicCAS(p.status, 0, MLA_ERR_DEVICE_CHECK);
        return n;
    };
    auto claim = [&](int t, int at, int x) {  // token t has tiles [at, at + x) of the line
        if (at <= t_lo && t_lo < at + x) {
            sh_token = t;
            sh_tile = t_lo - at;
        }
    };
    if (p.tokens <= kScoreThreads) {
        const int x = tid < p.tokens ? tiles_at(tid) : 0;
        int line;
        const int at = block_scan(x, line);
        cut(line);
        claim(tid, at, x);
    } else {
        int mine = 0;
        for (int t = tid; t < p.tokens; t += kScoreThreads) mine += tiles_at(t);
        int line;
        block_scan(mine, line);
        cut(line);
        for (int t0 = 0, base = 0; t0 < p.tokens && base <= t_lo; t0 += kScoreThreads) {
            const int x = t0 + tid < p.tokens ? tiles_of(seen_by(p, t0 + tid)) : 0;
            int total;
            const int at = base + block_scan(x, total);
            claim(t0 + tid, at, x);
            base += total;
        }
    }
    __syncthreads();
    const int n_here = t_hi - t_lo;
    uint32_t tmem = 0;

    // Position on the line: token (p.tokens: none), first page of its tile, pages that the token sees, the
    // token's row of the block table.
    struct Place {
        int token, j0, pages;
        const int32_t* table;
    };
    const Place none{p.tokens, 0, 0, nullptr};
    auto place_of = [&](int token, int tile) {
        if (token >= p.tokens) return none;
        return Place{token, tile * kTile, pages_of(seen_by(p, token)),
                     p.block_table + static_cast<size_t>(token / p.s_q) * p.max_blocks};
    };
    auto next_of = [&](const Place& a) {
        if (a.j0 + kTile < a.pages) return Place{a.token, a.j0 + kTile, a.pages, a.table};
        Place b = place_of(a.token + 1, 0);
        while (b.token < p.tokens && b.pages == 0) b = place_of(b.token + 1, 0);
        return b;
    };
    const int my_row = 8 * warp + (lane & 7);  // lanes 0-7: the row of a tile whose page this lane looks up
    // Its block-table entry (kNoRow past the token's pages), read a tile before checked() looks at it, so
    // that nothing waits for it; and the page: -1 for no row.
    constexpr int kNoRow = -0x7fffffff - 1;
    auto entry_at = [&](const Place& a) {
        const int j = a.j0 + my_row;
        return lane < 8 && j < a.pages ? __ldg(a.table + j) : kNoRow;
    };
    auto checked = [&](int entry, const Place& a) {
        if (lane >= 8 || a.j0 + my_row >= a.pages) return -1;
        if (entry < 0 || entry >= p.num_blocks) {
            if (p.status) atomicCAS(p.status, 0, MLA_ERR_DEVICE_CHECK);
            return 0;
        }
        return entry;
    };
    constexpr int kWords = kD / 16;  // 16-byte words of a row
    // Word c of row r in a tile of 64-byte swizzled rows: word c % 4 of box c / 4 at (c % 4) ^ ((r / 2) % 4).
    auto word_at = [](int r, int c) { return (c >> 2) * kKeyBoxBytes + r * 64 + (((c & 3) ^ ((r >> 1) & 3)) << 4); };
    // An instruction copies 16 words of two rows: both rows' 64 bytes of a box fill one 128-byte line of
    // shared memory (32 words of one row meet on half the banks, eight ways).
    const int half_row = lane >> 4, half_word = lane & 15;
    auto load_tile = [&](int stage, int page) {  // this warp's 8 rows; lane l < 8 gives the page of row l
        const uint32_t dst = s_base + L::kOffK + stage * L::kTileBytes;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const int pg = __shfl_sync(0xffffffffu, page, k + half_row), r = 8 * warp + k + half_row;
            const int8_t* src = p.keys + static_cast<size_t>(max(pg, 0)) * kD + 16 * half_word;
            cp_async16(dst + word_at(r, half_word), src, pg >= 0);
            cp_async16(dst + word_at(r, 16 + half_word), src + 256, pg >= 0);
        }
        if constexpr (kWords > 32) {  // the last 4 words of the 8 rows, one a lane
            static_assert(kWords == 36 || kWords == 32, "four words left over");
            const int pg = __shfl_sync(0xffffffffu, page, lane >> 2), c = 32 + (lane & 3);
            cp_async16(dst + word_at(8 * warp + (lane >> 2), c), p.keys + static_cast<size_t>(max(pg, 0)) * kD + 16 * c, pg >= 0);
        }
        cp_async_commit();
    };
    const int ncols = (p.h_q + 31) & ~31;
    auto load_queries = [&](int token, int buf) {
        // In the layout of the tiles, 8 rows a warp; rows past the last head are zero.
        const int8_t* base = p.q8 + static_cast<size_t>(token) * p.h_q * kD;
        if (8 * warp < ncols) {
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const int h = 8 * warp + k + half_row;
                const int8_t* src = base + static_cast<size_t>(h < p.h_q ? h : 0) * kD + 16 * half_word;
                cp_async16(s_base + L::kOffQ + word_at(h, half_word), src, h < p.h_q);
                cp_async16(s_base + L::kOffQ + word_at(h, 16 + half_word), src + 256, h < p.h_q);
            }
            if constexpr (kWords > 32) {
                const int h = 8 * warp + (lane >> 2), c = 32 + (lane & 3);
                cp_async16(s_base + L::kOffQ + word_at(h, c), base + static_cast<size_t>(h < p.h_q ? h : 0) * kD + 16 * c, h < p.h_q);
            }
        }
        if (tid < ncols) qscale[buf][tid] = tid < p.h_q ? __ldcg(p.q8_scales + static_cast<size_t>(token) * p.h_q + tid) : 0.f;
        cp_async_commit();
    };
    const uint32_t idesc = instr_desc_i8(kTile, ncols);
    const bool elected = elect_one();
    const uint64_t q_desc = smem_desc(s_base + L::kOffQ, 16, 512, kLayoutSW64);
    const uint64_t k_desc = smem_desc(s_base + L::kOffK, 16, 512, kLayoutSW64);
    auto products = [&](auto stage_c) {
        constexpr int kStage = decltype(stage_c)::value;  // addresses differ by constants only: quick to issue
#pragma unroll
        for (int ks = 0; ks < 2 * L::kBoxes; ++ks) {  // 32 columns per step
            constexpr uint32_t kA = (kStage * L::kTileBytes) >> 4;
            const uint32_t off = ((ks >> 1) * kKeyBoxBytes + (ks & 1) * 32) >> 4;
            mma_i8_ss(tmem + 128 * kStage, k_desc + kA + off, q_desc + off, idesc, ks > 0 ? 1u : 0u);
        }
        mma_commit(bar);
    };
    auto start_products = [&](int stage) {  // one lane of warp 0
        if (warp != 0) return;
        if (stage == 0) {
            if (elected) products(std::integral_constant<int, 0>{});
        } else {
            if (elected) products(std::integral_constant<int, 1>{});
        }
        __syncwarp();
    };

    // (What is read before grid_dependency_wait was written before the quantizing kernel started.)
    bool ok = true;
    if (n_here > 0) {
        Place cur = place_of(sh_token, sh_tile), nxt = n_here > 1 ? next_of(cur) : none;
        Place after = n_here > 2 ? next_of(nxt) : none;
        const int entry_cur = entry_at(cur), entry_nxt = entry_at(nxt);
        int entry_after = entry_at(after);
        const int page_cur = checked(entry_cur, cur);
        load_tile(0, page_cur);
        int page_nxt = checked(entry_nxt, nxt);
        if (warp == 0) {  // (its latency behind the first copies)
            tmem_alloc(smem_addr(tmem_slot), 256);
            tmem_relinquish();
        }
        float scale_cur = page_cur >= 0 ? __ldg(p.scales + page_cur) : 0.f;
        grid_dependency_wait();
        load_queries(cur.token, 0);
        int qbuf = 0;
        if (n_here > 1) {
            load_tile(1, page_nxt);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        fence_proxy_async_smem();  // this thread's copies, before the tensor core reads them
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
        start_products(0);
        for (int i = 0; i < n_here; ++i) {
            const int stage = i & 1;
            const bool more = i + 1 < n_here;
            const Place third = i + 3 < n_here ? next_of(after) : none;
            const int entry_third = entry_at(third);
            const int page_after = checked(entry_after, after);
            const float scale_nxt = page_nxt >= 0 ? __ldg(p.scales + page_nxt) : 0.f;
            ok = mbar_wait_bounded(bar, i & 1);
            ok = __syncthreads_and(ok) != 0;  // (and the last tile's maxima are taken)
            if (!ok) break;
            const bool new_token = more && nxt.token != cur.token;
            const int qb = qbuf;
            if (new_token) load_queries(nxt.token, qbuf ^= 1);
            if (i + 2 < n_here) {
                load_tile(stage, page_after);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
            if (more) {
                fence_proxy_async_smem();
                tc_fence_before();
                __syncthreads();
                tc_fence_after();
                start_products(stage ^ 1);
            }
            tc_fence_after();
            // Thread (lane quarter, column group): its page's maximum over 32 heads.
            const int row = 32 * (warp & 3) + lane, cg = warp >> 2;
            if (32 * cg < ncols) {
                uint32_t v[32];
                tmem_ld32(tmem + 128 * stage + 32 * cg + (static_cast<uint32_t>(32 * (warp & 3)) << 16), v);
                tmem_wait_ld();
                reg_fence(v);
                float m = -INFINITY;
                const int real = p.h_q - 32 * cg;  // heads of this group
                const float4* qs = reinterpret_cast<const float4*>(qscale[qb] + 32 * cg);
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const float4 q4 = qs[c / 4];
                    const float x0 = __fmul_rn(static_cast<float>(static_cast<int>(v[c])), q4.x);
                    const float x1 = __fmul_rn(static_cast<float>(static_cast<int>(v[c + 1])), q4.y);
                    const float x2 = __fmul_rn(static_cast<float>(static_cast<int>(v[c + 2])), q4.z);
                    const float x3 = __fmul_rn(static_cast<float>(static_cast<int>(v[c + 3])), q4.w);
                    if (c + 4 <= real) {
                        m = fmaxf(m, fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)));
                    } else {
                        if (c < real) m = fmaxf(m, x0);
                        if (c + 1 < real) m = fmaxf(m, x1);
                        if (c + 2 < real) m = fmaxf(m, x2);
                    }
                }
                red[stage][cg][row] = m;
            }
            tc_fence_before();
            __syncthreads();
            if (lane < 8) {
                const int j = cur.j0 + my_row, n_pages = cur.pages;
                float m = red[stage][0][my_row];
                for (int c = 1; 32 * c < ncols; ++c) m = fmaxf(m, red[stage][c][my_row]);
                float s = __fmul_rn(m, scale_cur);
                // finite, so that nothing beats a page that is always in
                s = s == s ? fminf(fmaxf(s, -FLT_MAX), FLT_MAX) : -FLT_MAX;
                if (j < p.first || j >= n_pages - p.last) s = INFINITY;
                if (j < n_pages) p.scores[static_cast<size_t>(cur.token) * p.max_blocks + j] = s;
            }
            cur = nxt;
            nxt = after;
            after = third;
            scale_cur = scale_nxt;
            page_nxt = page_after;
            entry_after = entry_third;
        }
    }
    if (n_here <= 0) grid_dependency_wait();  // no CTA, and so not the grid, ends before the quantizing one
    if (!ok) {
        // A product that never completed: say so, give the copies and it time to end, and leave.
        if (tid == 0 && p.status) atomicCAS(p.status, 0, MLA_ERR_TIMEOUT);
        cp_async_wait<0>();
        const uint64_t start = global_timer_ns();
        while (global_timer_ns() - start < 50000000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && n_here > 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// Selection: one CTA per token.  What is searched for is the topn-th largest score as an
// order-preserving 32-bit pattern; the pages above it are in, and of those equal to it the first.
// Up to 8,192 pages, in registers: the scores that compete are counted in 1,024 bins between the smallest
// and the largest of them, a suffix sum finds the bin that the searched one is in, and the few scores
// of that bin rank one another: 4 exchanges between warps, about 1 us.  Where a bin holds too many
// (equal scores), and for more pages, two bits of the pattern a round: each counts the scores at or
// above three candidates; 16 rounds, 4.1 us.
// Thread i holds scores [i * kPer, (i + 1) * kPer), so prefix sums give the pages in order and ties to
// the lower.  kPer 0: scores are read again each round.
constexpr int kSelectThreadsSmall = 256, kSelectPerSmall = 8;    // up to 2,048 pages
constexpr int kSelectThreadsLarge = 1024, kSelectPerLarge = 8;   // up to 8,192

template <int kThreads, int kPer>
__global__ void __launch_bounds__(kThreads) mla_select_pages_kernel(const SelectParams p)
{
    constexpr int kWarps = kThreads / 32;
    __shared__ int part[2][3][kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t = blockIdx.x;
    // What the selection reads beside the scores is older than the quantizing kernel's start: it is
    // fetched while the scores are still being computed.
    const int sees = seen_by(p, t);
    const int n = pages_of(sees);
    const int per = kPer > 0 ? kPer : (n + kThreads - 1) / kThreads;
    const float* scores = p.scores + static_cast<size_t>(t) * p.max_blocks;
    const int32_t* table = p.block_table + static_cast<size_t>(t / p.s_q) * p.max_blocks;
    int32_t* out = p.out_table + static_cast<size_t>(t) * p.topn;
    const int keep = min(n, p.topn);
    int32_t mine[kPer > 0 ? kPer : 1];  // this thread's pages
    if constexpr (kPer > 0) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) mine[k] = tid * kPer + k < n ? __ldg(table + tid * kPer + k) : 0;
    }
    grid_dependency_wait();
    for (int i = keep + tid; i < p.topn; i += kThreads) out[i] = -1;
    if (tid == 0) p.out_lens[t] = n > 0 ? (keep - 1) * kPage + (sees - (n - 1) * kPage) : 0;
    if (n <= p.topn) {
        for (int i = tid; i < n; i += kThreads) out[i] = table[i];
        return;
    }
    // Order-preserving pattern: larger score, larger number; 0 past the pages (below every score).
    auto pattern = [&](int j) -> uint32_t {
        if (j >= n) return 0u;
        const uint32_t u = __float_as_uint(__ldcg(scores + j) + 0.0f);  // -0 counts as 0
        return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    };
    uint32_t key[kPer > 0 ? kPer : 1];
    if constexpr (kPer > 0) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) key[k] = pattern(tid * kPer + k);
    }
    auto get = [&](int k) -> uint32_t {
        if constexpr (kPer > 0)
            return key[k];
        else
            return pattern(tid * per + k);
    };
    int buf = 0;
    // Sums over the block.  With kPer the counts are at most 8,192: two share a word.
    auto sum3 = [&](int a, int b, int c, int& ta, int& tb, int& tc) {
        const bool in = lane < kWarps;
        if constexpr (kPer > 0) {
            const unsigned ab = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(a) | (static_cast<unsigned>(b) << 16));
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == 0) {
                part[buf][0][warp] = static_cast<int>(ab);
                part[buf][1][warp] = c;
            }
            __syncthreads();
            const unsigned t2 = __reduce_add_sync(0xffffffffu, in ? static_cast<unsigned>(part[buf][0][lane]) : 0u);
            tc = __reduce_add_sync(0xffffffffu, in ? part[buf][1][lane] : 0);
            ta = static_cast<int>(t2 & 0xffffu);
            tb = static_cast<int>(t2 >> 16);
        } else {
            a = __reduce_add_sync(0xffffffffu, a);
            b = __reduce_add_sync(0xffffffffu, b);
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == 0) {
                part[buf][0][warp] = a;
                part[buf][1][warp] = b;
                part[buf][2][warp] = c;
            }
            __syncthreads();
            ta = __reduce_add_sync(0xffffffffu, in ? part[buf][0][lane] : 0);
            tb = __reduce_add_sync(0xffffffffu, in ? part[buf][1][lane] : 0);
            tc = __reduce_add_sync(0xffffffffu, in ? part[buf][2][lane] : 0);
        }
        buf ^= 1;
    };
    uint32_t thr = 0;  // the largest pattern with at least topn scores at or above it
    bool found = false;
    if constexpr (kPer > 0) {
        // Two 16-bit counts a word: such a block then fits beside one of the scoring kernel's, to start early.
        constexpr int kBins = 1024, kEach = kBins / kThreads, kMostRanked = 128;
        constexpr uint32_t kInf = 0xff800000u;  // pattern of the pages that are always in; no other has it
        __shared__ uint32_t hist[kBins / 2];
        auto count_of = [&](int b) { return static_cast<int>((hist[b >> 1] >> (16 * (b & 1))) & 0xffffu); };
        __shared__ uint32_t ranked[kMostRanked];
        __shared__ uint32_t sh_thr;
        __shared__ int sh_bin, sh_need, sh_ranked;
        auto value = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k); };
        uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (key[k] != 0u && key[k] != kInf) {
                lo = min(lo, key[k]);
                hi = max(hi, key[k]);
            }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            part[0][0][warp] = static_cast<int>(lo);
            part[0][1][warp] = static_cast<int>(hi);
        }
        for (int k = tid; k < kBins / 2; k += kThreads) hist[k] = 0;
        if (tid == 0) sh_ranked = 0;
        __syncthreads();
        lo = __reduce_min_sync(0xffffffffu, lane < kWarps ? static_cast<uint32_t>(part[0][0][lane]) : 0xffffffffu);
        hi = __reduce_max_sync(0xffffffffu, lane < kWarps ? static_cast<uint32_t>(part[0][1][lane]) : 0u);
        const int need = p.topn - p.first - p.last;  // of the competing scores (n > topn: some compete)
        // Halves, so that the range is finite.  Each step is monotonic, so a larger score is in no lower bin.
        const float base = 0.5f * value(lo), width = 0.5f * value(hi) - base, inv = (kBins - 1) / width;
        if (need == 0) {
            thr = kInf;
            found = true;
        } else if (width > 0.f && inv < FLT_MAX && inv > 0.f) {  // (the same for every thread)
            int bin[kPer];
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const bool in = key[k] != 0u && key[k] != kInf;
                bin[k] = in ? min(kBins - 1, static_cast<int>((0.5f * value(key[k]) - base) * inv)) : -1;
                if (in) atomicAdd(&hist[bin[k] >> 1], 1u << (16 * (bin[k] & 1)));
            }
            __syncthreads();
            // scores in this thread's bins and in the threads' above
            int own = 0;
#pragma unroll
            for (int k = 0; k < kEach; ++k) own += count_of(tid * kEach + k);
            int suffix = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_down_sync(0xffffffffu, suffix, o);
                if (lane + o < 32) suffix += y;
            }
            if (lane == 0) part[1][0][warp] = suffix;
            __syncthreads();
            int more = 0;
            for (int w = warp + 1; w < kWarps; ++w) more += part[1][0][w];
            int above = more + suffix - own;  // in the bins above this thread's
            if (above < need && need <= above + own) {
#pragma unroll
                for (int k = kEach - 1; k >= 0; --k) {
                    const int c = count_of(tid * kEach + k);
                    if (above < need && need <= above + c) {
                        sh_bin = tid * kEach + k;
                        sh_need = need - above;
                    }
                    above += c;
                }
            }
            __syncthreads();
            const int the_bin = sh_bin, rank = sh_need, many = count_of(the_bin);
            if (many <= kMostRanked) {
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    if (bin[k] == the_bin) ranked[atomicAdd(&sh_ranked, 1)] = key[k];
                __syncthreads();
                // the rank-th largest of them (equal ones give the same answer)
                if (tid < many) {
                    const uint32_t x = ranked[tid];
                    int greater = 0, equal = 0;
                    for (int c = 0; c < many; ++c) {
                        greater += ranked[c] > x;
                        equal += ranked[c] == x;
                    }
                    if (greater < rank && rank <= greater + equal) sh_thr = x;
                }
                __syncthreads();
                thr = sh_thr;
                found = true;
            }
        }
        __syncthreads();  // part may be written again
    }
    for (int bit = 30; bit >= 0 && !found; bit -= 2) {
        const uint32_t c1 = thr | (1u << bit), c2 = thr | (2u << bit), c3 = thr | (3u << bit);
        int a = 0, b = 0, c = 0;
        if constexpr (kPer > 0) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                a += key[k] >= c1;
                b += key[k] >= c2;
                c += key[k] >= c3;
            }
        } else {
            for (int k = 0; k < per; ++k) {
                const uint32_t x = get(k);  // (0 past the pages: below every candidate)
                a += x >= c1;
                b += x >= c2;
                c += x >= c3;
            }
        }
        int ta, tb, tc;
        sum3(a, b, c, ta, tb, tc);
        thr = tc >= p.topn ? c3 : (tb >= p.topn ? c2 : (ta >= p.topn ? c1 : thr));
    }
    int above = 0, equal = 0;
#pragma unroll (kPer > 0 ? kPer : 1)
    for (int k = 0; k < per; ++k) {
        const uint32_t x = get(k);
        above += x > thr;
        equal += x == thr;
    }
    // exclusive prefix sums of both over the threads (in page order)
    auto scan = [&](int x, int& before, int& total) {
        int incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) part[buf][0][warp] = incl;
        __syncthreads();
        int b = 0;
        total = 0;
        for (int w = 0; w < kWarps; ++w) {
            const int v = part[buf][0][w];
            if (w < warp) b += v;
            total += v;
        }
        before = b + incl - x;
        buf ^= 1;
    };
    int above_before, above_total, equal_before, equal_total;
    scan(above, above_before, above_total);
    scan(equal, equal_before, equal_total);
    const int room = p.topn - above_total;  // how many of the equal ones are in: the first
    int at = above_before + min(equal_before, room);
#pragma unroll (kPer > 0 ? kPer : 1)
    for (int k = 0; k < per; ++k) {
        const uint32_t x = get(k);
        const bool in = x > thr || (x == thr && equal_before < room);
        equal_before += x == thr;
        if (in) {
            if constexpr (kPer > 0)
                out[at++] = mine[k];
            else
                out[at++] = table[tid * per + k];
        }
    }
}

template <int kD, bool kFp16>
static cudaError_t launch_scores(int grid, cudaStream_t st, const SelectParams& prm)
{
    auto kern = mla_score_pages_kernel<kD, kFp16>;
    constexpr int smem = ScoreLayout<kD>::kBytes;
    static PerDeviceOnce configured;
    cudaError_t e = configured.run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    const long long rows = static_cast<long long>(prm.tokens) * prm.h_q;
    constexpr int kWarps = kQuantThreads / 32;
    mla_quantize_queries_kernel<kD, kFp16><<<static_cast<unsigned>((rows + kWarps - 1) / kWarps), kQuantThreads, 0, st>>>(prm);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    programmatic_launch(cfg, attr, dim3(grid), dim3(kScoreThreads), smem, st);
    return cudaLaunchKernelEx(&cfg, kern, prm);
}

}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_select_workspace_bytes(int batch, int s_q, int h_q, int d_qk, int max_blocks_per_seq)
{
    if (batch < 0 || s_q <= 0 || h_q <= 0 || d_qk <= 0 || max_blocks_per_seq <= 0) return 0;
    // queries in 8 bits, their scales, the scores
    const double most = static_cast<double>(batch) * s_q * (static_cast<double>(h_q) * (d_qk + 4.0) + 4.0 * max_blocks_per_seq);
    if (most >= 1e15) return 0;
    const size_t tokens = static_cast<size_t>(batch) * s_q;
    return tokens * (static_cast<size_t>(h_q) * (d_qk + 4) + 4 * static_cast<size_t>(max_blocks_per_seq)) + 256;
}

mla_status mla_select_pages(const void* q, int batch, int s_q, int h_q, int d_qk, int dtype, const int8_t* page_keys,
                            const float* page_scales, int num_blocks, const int32_t* block_table, int max_blocks_per_seq,
                            const int32_t* cache_seqlens, int causal, int topn, int n_first, int n_last,
                            int32_t* page_table, int32_t* page_seqlens, void* workspace, size_t workspace_bytes,
                            int32_t* device_status, void* stream)
{
    if (batch < 0 || s_q <= 0 || h_q <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || (causal != 0 && causal != 1))
        return MLA_ERR_INVALID_ARG;
    if (dtype != MLA_BF16 && dtype != MLA_FP16) return dtype == MLA_BF16_FP8KV ? MLA_ERR_UNSUPPORTED : MLA_ERR_INVALID_ARG;
    if (n_first < 0 || n_last < 1 || topn < 1 || n_first > topn || n_last > topn - n_first) return MLA_ERR_INVALID_ARG;
    if ((d_qk != 576 && d_qk != 512) || h_q > kMaxHeads) return MLA_ERR_UNSUPPORTED;
    // rows of a cache, and of a block table (topn columns of the chosen pages' one), are counted in int32
    constexpr long long kMostRows = 1ll << 31;
    if (static_cast<long long>(num_blocks) * kPage >= kMostRows || static_cast<long long>(max_blocks_per_seq) * kPage >= kMostRows ||
        static_cast<long long>(topn) * kPage >= kMostRows)
        return MLA_ERR_UNSUPPORTED;
    const long long tokens = static_cast<long long>(batch) * s_q;
    // the line of tiles is counted in int32
    if (tokens * ((max_blocks_per_seq + kTile - 1) / kTile) >= (1ll << 31) || tokens >= (1ll << 31) / h_q) return MLA_ERR_UNSUPPORTED;
    if (batch == 0) return MLA_OK;
    if (!q || !page_keys || !page_scales || !block_table || !cache_seqlens || !page_table || !page_seqlens || !workspace)
        return MLA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) & 15) || (reinterpret_cast<uintptr_t>(page_keys) & 15) ||
        (reinterpret_cast<uintptr_t>(workspace) & 15))
        return MLA_ERR_INVALID_ARG;
    if (workspace_bytes < mla_select_workspace_bytes(batch, s_q, h_q, d_qk, max_blocks_per_seq)) return MLA_ERR_WORKSPACE;
    int sms = 0;
    if (!sm_count(&sms)) return MLA_ERR_CUDA;
    SelectParams prm{};
    prm.q = static_cast<const uint8_t*>(q);
    prm.keys = page_keys;
    prm.scales = page_scales;
    prm.block_table = block_table;
    prm.seqlens = cache_seqlens;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    prm.q8 = reinterpret_cast<int8_t*>(ws);
    prm.q8_scales = reinterpret_cast<float*>(ws + static_cast<size_t>(tokens) * h_q * d_qk);  // d_qk: a multiple of 16
    prm.scores = prm.q8_scales + static_cast<size_t>(tokens) * h_q;
    prm.out_table = page_table;
    prm.out_lens = page_seqlens;
    prm.status = device_status;
    prm.tokens = static_cast<int>(tokens);
    prm.s_q = s_q;
    prm.h_q = h_q;
    prm.max_blocks = max_blocks_per_seq;
    prm.num_blocks = num_blocks;
    prm.topn = topn;
    prm.first = n_first;
    prm.last = n_last;
    prm.causal = causal;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const long long most = tokens * ((max_blocks_per_seq + kTile - 1) / kTile);
    const int grid = most < sms ? static_cast<int>(most) : sms;
    cudaError_t e;
    if (d_qk == 576)
        e = dtype == MLA_FP16 ? launch_scores<576, true>(grid, st, prm) : launch_scores<576, false>(grid, st, prm);
    else
        e = dtype == MLA_FP16 ? launch_scores<512, true>(grid, st, prm) : launch_scores<512, false>(grid, st, prm);
    if (e != cudaSuccess) return MLA_ERR_CUDA;
    const bool small = max_blocks_per_seq <= kSelectThreadsSmall * kSelectPerSmall;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    programmatic_launch(cfg, attr, dim3(static_cast<unsigned>(tokens)), dim3(small ? kSelectThreadsSmall : kSelectThreadsLarge), 0, st);
    if (small)
        e = cudaLaunchKernelEx(&cfg, mla_select_pages_kernel<kSelectThreadsSmall, kSelectPerSmall>, prm);
    else if (max_blocks_per_seq <= kSelectThreadsLarge * kSelectPerLarge)
        e = cudaLaunchKernelEx(&cfg, mla_select_pages_kernel<kSelectThreadsLarge, kSelectPerLarge>, prm);
    else
        e = cudaLaunchKernelEx(&cfg, mla_select_pages_kernel<kSelectThreadsLarge, 0>, prm);
    return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
