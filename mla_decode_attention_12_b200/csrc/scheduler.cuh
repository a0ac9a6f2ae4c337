// Tile scheduler: splits the decode work of a batch into `num_parts` contiguous
// ranges of equal cost, one per two-SM cluster of the split-KV kernel.
//
// "FlashMLA" usage page (deepep.org): get_mla_metadata analyses the sequence
// lengths once per decoding step and returns tile_scheduler_metadata and
// num_splits, reused by every layer; its Tile Scheduler "distributes work across
// GPU resources" and balances variable-length sequences ("optimized for
// variable-length sequence serving", sourcepulse summary).  The pages do not
// print the algorithm or the metadata format; this one is our own.
//
// Work units.  A "virtual batch" vb = g * batch + b is request b restricted to query
// rows [128 g, 128 g + 128) of its s_q * h_q rows.  The numbering is group-major: row
// group 0 of every request comes before row group 1 of any, so on the line below the
// groups of one request lie half a line (for two groups) apart, and the partitions that
// cover them stream the same pages at about the same time (the second read hits L2).  Every chunk (one
// partition's share of one virtual batch) costs F units of overhead (the output
// epilogue, refilling the pipeline) plus one unit per 64-token page: F = kFixedCost
// for the paged decode (kFixedCostFp8 over an FP8 cache, whose pages take about twice
// as long), kFixedCostSparse for the sparse calls, whose "pages" of 64 gathered
// entries cost two to three times a contiguous page.
// Lay the virtual batches on a line: vb takes F units followed by its pages,
// starting at C[vb] = sum of the costs before it; W is the total.  A partition
// that starts inside a virtual batch's pages opens one more chunk than the line
// shows, so it gets F units fewer of the line: with D = ceil((W - F) / num_parts),
// partition 0 takes the line units [0, F + D) and partition p >= 1 the units
// [F + p D, F + (p + 1) D); each partition's cost (pages + F per chunk) is then
// at most F + D.  D is at least F: a small batch leaves the last partitions empty rather
// than cutting its sequences into pieces smaller than a chunk's overhead.  A unit position x maps to the page position (vb, blk) with vb
// the virtual batch whose span holds x and blk = clamp(x - C[vb] - F, 0,
// pages(vb)); partition p covers the page positions from map(start p) up to
// map(start p+1).  A virtual batch whose pages are cut by partition starts is
// split; every partition computes its range on its own, so the device version
// is one thread per partition.
//
// Output:
//   md[p * 8 + 0..4] = begin_vb, begin_blk, end_vb, end_blk, begin_split
//     partition p covers the positions (vb, blk) with
//     (begin_vb, begin_blk) <= (vb, blk) < (end_vb, end_blk) in lexicographic
//     order; a virtual batch with no pages is the single position (vb, 0).
//     begin_split is the split index of partition p's first chunk within
//     begin_vb (later chunks of the partition start their virtual batch, index 0).
//   num_splits[vb] = sum of split counts of virtual batches before vb
//     (num_splits[NV] = total), so vb has num_splits[vb+1] - num_splits[vb] splits
//     and its k-th split result goes to workspace slot num_splits[vb] + k.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MLA_HD __host__ __device__
#else
#define MLA_HD
#endif

namespace mla {

constexpr int kPage = 64;
constexpr int kRowsPerGroup = 128;
constexpr int kFixedCost = 12;       // per-chunk overhead in page units (epilogue, pipeline refill), tuned on B200
constexpr int kFixedCostFp8 = 6;     // the same for the paged decode over an FP8 cache, tuned on B200
constexpr int kFixedCostSparse = 4;  // the same for the sparse decode and prefill, tuned on B200
constexpr int kMdInts = 8;

// Ragged runs of query tokens (chunks of prompts beside decode steps): run b is the query tokens
// [cu[b], cu[b + 1]), its rows (tokens x heads) are cut into groups of 128, and a group is a virtual
// batch.  On the cost line groups 0, P, 2 P, ... come first, then 1, P + 1, ... (P partitions, groups counted
// run by run), so that at any time the partitions work on neighbouring groups, which read the same
// pages: the second read hits L2.  (Run by run, a partition reads a run's pages once for each of its
// groups, and all runs are open at once.  Same box, run by run against this order: four prompts' pieces
// 4993 and 4820 us, eight over an FP8 cache 763 and 713, 32 runs of 14 groups over 8 MB each 1188 and 1153.)  One row of the group table per virtual batch, in line order:
enum VarField : int {
    kVarReq = 0,     // the run (request)
    kVarRow0 = 1,    // its first query row in the call's total_q * h_q rows
    kVarRows = 2,    // its rows (at most 128)
    kVarLimit = 3,   // cached rows that its last token sees: its pages end there
    kVarSeen = 4,    // a row of token t (of the call's tokens) sees clamp(kVarSeen + t, 0, kVarLen) cached rows
    kVarLen = 5,     // the request's cached rows
    kVarSplits = 6,  // partitions that share it
    kVarInts = 8
};

// Group (counted run by run) at place i of the line.
MLA_HD inline int group_on_line(int i, int nv, int num_parts)
{
    const int q = nv / num_parts, longer = nv % num_parts;  // `longer` classes have q + 1 groups, the others q
    const int head = longer * (q + 1);
    if (i < head) return (i % (q + 1)) * num_parts + i / (q + 1);
    return ((i - head) % q) * num_parts + longer + (i - head) / q;
}

// Visible rows of token `tok` (of the call's tokens) of a run of tokens [t0, t1) over len cached
// rows: the causal mask is aligned to the bottom right.
MLA_HD inline int run_seen(int t1, int len, bool causal)
{
    return causal ? len - t1 + 1 : 0x40000000;
}

MLA_HD inline int clamp_seen(long long seen, int len)
{
    return seen < 0 ? 0 : (seen < len ? static_cast<int>(seen) : len);
}

constexpr int kVarMostRows = 1 << 30;  // no cache holds as many rows; page counts stay in 32 bits

// Cached rows that the groups of a run of tokens [t0, t1) read (its last token sees them all).
MLA_HD inline int run_reads(int t0, int t1, int len)
{
    return t1 <= t0 || len < 0 ? 0 : (len < kVarMostRows ? len : kVarMostRows);
}

// Group g of run b = tokens [t0, t1): its row of the table (kVarSplits = 1).
MLA_HD inline void fill_group(int32_t* gr, int b, int g, int t0, int t1, int len, int h_q, bool causal)
{
    if (len > kVarMostRows) len = kVarMostRows;
    const int row0 = t0 * h_q + g * kRowsPerGroup, end = t1 * h_q;
    const int rows = end - row0 < kRowsPerGroup ? end - row0 : kRowsPerGroup;
    const int seen = run_seen(t1, len, causal);
    gr[kVarReq] = b;
    gr[kVarRow0] = row0;
    gr[kVarRows] = rows;
    gr[kVarLimit] = clamp_seen(static_cast<long long>(seen) + (row0 + rows - 1) / h_q, len);
    gr[kVarSeen] = seen;
    gr[kVarLen] = len;
    gr[kVarSplits] = 1;
    gr[7] = 0;
}

MLA_HD inline int row_groups(int heads_per_kv) { return (heads_per_kv + kRowsPerGroup - 1) / kRowsPerGroup; }

MLA_HD inline int pages_of(int seqlen) { return seqlen <= 0 ? 0 : (seqlen + kPage - 1) / kPage; }

// Request and row group of virtual batch vb (group-major numbering, batch requests).
MLA_HD inline int vb_request(int vb, int batch) { return vb % batch; }
MLA_HD inline int vb_group(int vb, int batch) { return vb / batch; }

// Position on the page line of cost unit x.  C: exclusive prefix of the costs,
// nv entries; total: W; F: the per-chunk cost.  Returns (vb, blk) through the references.
MLA_HD inline void unit_to_page(long long x, const long long* C, const int32_t* pages, int nv, long long total,
                                int F, int& vb, int& blk)
{
    if (x >= total || nv == 0) {
        vb = nv;
        blk = 0;
        return;
    }
    if (x < 0) x = 0;
    int lo = 0, hi = nv - 1;  // largest v with C[v] <= x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (C[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    long long b = x - C[lo] - F;
    if (b < 0) b = 0;
    vb = lo;
    blk = static_cast<int>(b);  // < pages[lo]: positions at or past the span's end belong to lo + 1
    (void)pages;
}

// Range of partition p: md row.  C / pages: per virtual batch; F: the per-chunk cost.
MLA_HD inline void partition_range(int p, int num_parts, const long long* C, const int32_t* pages, int nv,
                                   long long total, int F, int32_t* m)
{
    long long D = (total - F + num_parts - 1) / num_parts;  // line units of a partition after its first F
    // A partition shorter than one chunk's overhead would cost more than it saves: small
    // batches use fewer partitions (the rest get empty ranges) instead of one-page splits.
    if (D < F) D = F;
    auto start = [&](int q) -> long long { return q == 0 ? 0 : F + static_cast<long long>(q) * D; };
    int bv, bb, ev, eb;
    unit_to_page(start(p), C, pages, nv, total, F, bv, bb);
    if (p == num_parts - 1) {
        ev = nv;
        eb = 0;
    } else {
        unit_to_page(start(p + 1), C, pages, nv, total, F, ev, eb);
    }
    m[0] = bv;
    m[1] = bb;
    m[2] = ev;
    m[3] = eb;
    m[4] = 0;
    m[5] = m[6] = m[7] = 0;
}

// Host reference of the whole schedule (the device kernel computes the same
// values in parallel).  Scratch: C [nv] and pages [nv].
inline void schedule_host(const int32_t* seqlens, int batch, int groups, int num_parts, int F, int32_t* md,
                          int32_t* num_splits, long long* C, int32_t* pages)
{
    const int nv = batch * groups;
    long long total = 0;
    for (int v = 0; v < nv; ++v) {
        pages[v] = pages_of(seqlens[vb_request(v, batch)]);
        C[v] = total;
        total += pages[v] + F;
    }
    for (int p = 0; p < num_parts; ++p) partition_range(p, num_parts, C, pages, nv, total, F, md + p * kMdInts);
    // split counts: 1 + number of partitions that start inside a virtual batch's pages
    for (int v = 0; v <= nv; ++v) num_splits[v] = 0;
    for (int p = 0; p < num_parts; ++p) {
        int32_t* m = md + p * kMdInts;
        if (m[1] > 0) {
            // index of this split = 1 + number of earlier mid-batch starts in the same vb
            int idx = 1;
            for (int q = p - 1; q >= 0 && md[q * kMdInts + 0] == m[0] && md[q * kMdInts + 1] > 0; --q) ++idx;
            m[4] = idx;
            num_splits[m[0] + 1] += 1;  // extra splits, accumulated below
        }
    }
    int acc = 0;
    for (int v = 0; v < nv; ++v) {
        const int extra = num_splits[v + 1];
        num_splits[v] = acc;
        acc += 1 + extra;
    }
    num_splits[nv] = acc;
}

// The same for ragged runs: group table, md rows and the rows that each run reads.  Scratch: C [groups].
inline void schedule_varlen_host(const int32_t* cu, const int32_t* seqlens, int batch, int h_q, bool causal, int num_parts,
                                 int F, int32_t* md, int32_t* groups, long long* C, int32_t* reads)
{
    int nv = 0;
    for (int b = 0; b < batch; ++b) reads[b] = run_reads(cu[b], cu[b + 1], seqlens[b]);
    for (int b = 0; b < batch; ++b) nv += row_groups((cu[b + 1] - cu[b]) * h_q);
    // C, until it holds the prefix sums: the place of each group on the line
    for (int i = 0; i < nv; ++i) C[group_on_line(i, nv, num_parts)] = i;
    for (int b = 0, v = 0; b < batch; ++b)
        for (int g = 0; g < row_groups((cu[b + 1] - cu[b]) * h_q); ++g, ++v)
            fill_group(groups + kVarInts * C[v], b, g, cu[b], cu[b + 1], seqlens[b], h_q, causal);
    long long total = 0;
    for (int i = 0; i < nv; ++i) {
        C[i] = total;
        total += pages_of(groups[static_cast<long long>(kVarInts) * i + kVarLimit]) + F;
    }
    for (int p = 0; p < num_parts; ++p) partition_range(p, num_parts, C, nullptr, nv, total, F, md + p * kMdInts);
    for (int p = 0; p < num_parts; ++p) {
        int32_t* m = md + p * kMdInts;
        if (m[1] > 0) {
            m[4] = 1;
            for (int q = p - 1; q >= 0 && md[q * kMdInts] == m[0] && md[q * kMdInts + 1] > 0; --q) ++m[4];
            ++groups[static_cast<long long>(kVarInts) * m[0] + kVarSplits];
        }
    }
}

}  // namespace mla
