// Attention of the newest tokens over the paged cache where groups of sequences
// share the pages that their tables begin with.
//
//   o = (sum_t e^{s_t - m} v_t) / sum_t e^{s_t - m}
// over a sequence's positions is joined from sums over any parts of them, so the
// shared positions of a group are taken once, with the rows of all its sequences
// (new tokens times query heads of the key head) as one matrix, and each
// sequence's own positions by themselves.  Four kernels in stream order, each
// launched ahead of the end of the one before, for which it waits ahead of its
// first read:
//
//   plan     one CTA reads offsets and lengths and cuts the work: how far each
//            group shares, tiles for the wide kernel, pieces for the narrow one
//   wide     groups (and trees of drafts) of more than 32 rows a key head, on
//            the tensor cores: this file
//   narrow   everything of up to 32 rows, over the plan's list, by the kernels of
//            bdla_cache.cu: a warp a piece for sequences of up to 16 rows, four
//            warps above; a sequence of one piece that shares nothing is finished
//            there
//   join     the sums of a row's pieces, in their order
//
// Everything that the cut depends on (group sizes, shared lengths, lengths) is on
// the device and changes from step to step under a captured graph, so the grids
// are sized from the tensors' shapes and the plan fills them.
//
// d = 128, 32 heads on 8, one token each: 256 sequences of up to 513 positions of
// their own behind 32768 shared ones 174 to 175 us, of it the wide kernel 107 (tensor
// cores; 1.44 PFLOP/s a further position, the whole-prompt forward's rate), the
// narrow one 51 (HBM, 5.7 TB/s), the join 12, the plan 7, one after the other but
// for their set-up; attention of each sequence by itself reads 34 GB, 4.2 ms.  16
// sequences behind 131072: 119 to 121 us, the wide kernel 91 of it (HBM, 5.9 TB/s).
// Where the narrow kernel read the plan's list without waiting for the wide one's
// end, as only the order of launches had it, the two took 170 and 116 us, and 64
// sequences behind 512 positions 36 for 40.  What is left: the plan's chain of
// latencies, the first tiles and the last sums of each kernel (about 45 us of the
// 174), and 168 registers a thread, beside which 48 to 68 bytes are spilled.
//
// Rounding: scores, weights, their sums and the sums of pieces are fp32; the
// weights are rounded to bf16 as they enter their product with the values, in both
// kernels, because the tensor cores take both operands in one type, and o once more
// at the end.  The error against 64 bits is then 1.7e-3 to 2.3e-3 of the norm, where
// weights of fp32 leave o's own 1.5e-3 to 1.7e-3.
#include <cudaTypedefs.h>

#include "bdla_attn_sm100.cuh"
#include "bdla_cache.cuh"

namespace bdla {

namespace {

using namespace sm100;
using namespace attn;
using namespace cache;

// Rows a key head up to which warp MMAs take a group, 16 at a time (32 rows: 20 us
// against 36 on the tensor cores behind 4096 positions, 82 against 73 behind 65536;
// 16 rows behind 65536: 61 against 73).  Where the batch has twice as many and no
// table more than kShortTable positions, the wide kernel is not launched at all (64
// rows: 17 to 21 us against 32 to 39 behind 64 to 3500 positions; behind 65536, 131
// against 75).
constexpr int kNarrowRows = 32, kShortTable = 4096;
constexpr int kWideTile = 256;    // rows of a CTA of the wide kernel
// What a change of rows costs the wide kernel, in tiles of 128 rows: its sums out,
// the next queries in, the first scores (64 sequences of 33 drafts, 490 us; 617
// with 2, 520 with 5, 512 with 16).
constexpr int kRun = 10;
constexpr int kSeen = INT32_MAX;  // "committed positions" where no new token is among those seen

// Elements of keys and values that a group has to save from being read again for
// its sums to be worth the joining (us with and without it, up to 401 positions of
// a sequence's own).  Where the tensor cores take the group and run for nothing
// else, their kernel's set-up has to be earned too: 64 sequences, 32 heads on 8 of
// 128: 35 against 32 with 17e6 elements (128 shared positions), 36 against 37 with
// 33e6, 40 against 42 with 66e6; 256 sequences: 72 against 58 with 33e6, 70 against
// 66 with 67e6, 70 against 71 with 100e6, 75 against 104 with 267e6.  Where warps
// take the group (8 sequences, 16 heads on 4: 16.4 against 16.7 with 1.8e6, 17.2
// against 19.2 with 15e6), and where the tensor cores run for the sequences' own
// positions anyway (more than kNarrowRows rows of one): 8 sequences of 17 tokens 30
// against 32 with 3.7e6 and 31 against 35 with 29e6, 29 of them 57 against 55 with 7e6
// and 70 against 82 with 117e6; with many rows and little shared it costs more than
// it gives (64 of 33 tokens, 151 against 129 with 17e6, 194 against 213 with 264e6),
// but the larger bound would leave short prompts of few trees unjoined.
constexpr int64_t kLeastWide = 64000000, kLeastNarrow = 2000000;

// What the wide kernel walks: positions first .. end - 1 of sequence b's table
// for the row blocks rb0 .. rb1 - 1 of the R rows from token tok0 on, times key
// heads.  A block of 256 rows is two row tiles of 128, the last one may be one;
// the blocks of an entry have `row_tiles` each.  On the line that the CTAs cut
// evenly a block and head is kRun and then nt tiles of 128 positions, which count
// row_tiles each; `base`: the line before the entry.
struct alignas(16) WideEntry {
    int base, b, tok0, R, first, end, len, nt, part, rb0, rb1, row_tiles;
};

// Where an entry's partial sums are.  wide (nt > 0): pieces follow from the cut of
// the line, whose blocks of two row tiles start at `base` and the last one of one
// row tile, block `full`, at `base1`; narrow: np pieces; np < 0: its rows are
// finished.
struct alignas(16) Parts {
    int base, nt, R, part, np, tok0, base1, full;
};

struct Head {
    int line;        // of the wide kernel
    int per_cta;     // of a CTA
    int2 list;       // pieces of the narrow kernel: the long ones from the front, the others from `y` on to the end
};

// Entries are the groups, then the sequences.
struct Plan {
    Head *head;
    WideEntry *wide;
    Parts *parts;
    Work *list;
    int *first_entry;   // of each CTA of the wide kernel
    int *group;         // of each sequence, -1: none
    int *scratch;       // of the plan, where shared memory is too small
    float *part_o, *part_ml;
};

struct Sizes {
    int B, T, G, Hk, D, n_groups;
    int ctas;            // of the wide kernel
    bool wide, own_wide; // the wide kernel runs; it takes the sequences' own positions too
    int narrow_tiles;    // rows of a narrow CTA, in 16
    int slots;           // narrow CTAs that the GPU holds
    float heads_per_slot;
    int extra;           // pieces of the narrow list beyond one for every block of rows
    int most;            // pieces of the narrow list
    int64_t rows;        // of partial sums
    int64_t least_wide, least_narrow;
};

// Integers that the plan keeps: offsets and shared lengths of the groups,
// lengths of all entries, the sequences' groups.
constexpr size_t plan_ints(int n_groups, int B) { return 3 * (size_t)n_groups + 2 * (size_t)B + 1; }

// Bounds of the plan.  Narrow: a piece size of at least the (block-weighted)
// positions over `extra` cuts at most `extra` pieces beyond the first of each
// block; sequences have one block, groups of at most 32 rows one or two, those of
// at most 64 in all no more than four beyond one each, and a group that shares has
// two sequences or more.  Wide: a block's tiles lie in
// row_tiles nt / per_cta + 2 CTAs at most; 256 rows for each of that for all of an
// entry's rows is at most 256 times its line, and the line at most ctas x per_cta.
Sizes sizes_of(const bdla_attn_dims &d, int n_groups, int64_t max_keys)
{
    Sizes s;
    s.B = d.B;
    s.T = d.T;
    s.G = d.Hq / d.Hk;
    s.Hk = d.Hk;
    s.D = d.d;
    s.n_groups = n_groups;
    const int64_t least = g_share_least.load();
    s.least_narrow = least < 0 ? kLeastNarrow : least;
    s.ctas = sm_count();
    const int64_t R = (int64_t)d.T * s.G, all = R * d.B;
    s.own_wide = R > kNarrowRows;
    s.least_wide = least < 0 && !s.own_wide ? kLeastWide : s.least_narrow;
    s.wide = s.own_wide || all > (max_keys > kShortTable ? kNarrowRows : 2 * kNarrowRows);
    s.narrow_tiles = R <= 16 ? 1 : 2;
    s.slots = s.ctas * (s.narrow_tiles == 1 ? (d.d == 128 ? 9 : 16) : d.d == 128 ? 3 : 4);
    s.heads_per_slot = (float)d.Hk / (float)s.slots;
    s.extra = 2 * ((s.slots + d.Hk - 1) / d.Hk);
    const int groups = n_groups < d.B / 2 ? n_groups : d.B / 2;
    s.most = s.own_wide ? 0 : d.B + 2 * groups + 4 + s.extra;
    s.rows = 0;
    if (s.wide)
        s.rows += 2 * all * d.Hk * (s.own_wide ? 2 : 1) + (int64_t)kWideTile * s.ctas;
    if (!s.own_wide)
        s.rows += (2 * all + (int64_t)kNarrowRows * s.extra) * d.Hk;
    return s;
}

size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

size_t carve(const Sizes &s, char *at, Plan *p)
{
    const size_t entries = (size_t)s.n_groups + s.B;
    size_t off = 0;
    const auto take = [&](auto *&ptr, size_t n) {
        ptr = reinterpret_cast<std::remove_reference_t<decltype(ptr)>>(at + off);
        off += aligned(n * sizeof(*ptr));
    };
    take(p->head, 1);
    take(p->wide, 2 * entries);
    take(p->parts, entries);
    take(p->list, (size_t)s.most);
    take(p->first_entry, (size_t)s.ctas);
    take(p->group, (size_t)s.B);
    take(p->scratch, plan_ints(s.n_groups, s.B));
    take(p->part_o, (size_t)s.rows * s.D);
    take(p->part_ml, (size_t)s.rows * 2);
    return off;
}

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = 512;
constexpr int kPlanEntries = 4000;   // whose offsets, groups and lengths fit into 48 KB of shared memory
constexpr int kLeastLine = 2 + kRun;   // of a wide CTA
constexpr int kFew = 4;               // pieces, or CTAs, of an entry that one lane writes
constexpr int kSizes = 8;            // piece sizes of the narrow kernel that are weighed: 128, 256 .. 16384 positions

__device__ __forceinline__ int tiles_of(int n) { return (int)(((uint32_t)n + BT - 1) / BT); }
__device__ __forceinline__ int over(int n, int size) { return (int)(((uint32_t)n + (uint32_t)size - 1) / (uint32_t)size); }

// What comes before an entry: line of the wide kernel, rows of partial sums,
// long and short pieces of the narrow list, entries of the wide one.
struct Sums {
    int tiles, rows, pieces, shorts, wides;
    __device__ __forceinline__ void add(const Sums &o)
    {
        tiles += o.tiles;
        rows += o.rows;
        pieces += o.pieces;
        shorts += o.shorts;
        wides += o.wides;
    }
    // Sums over this and the lower lanes.
    __device__ __forceinline__ Sums scanned() const
    {
        Sums s = *this;
#pragma unroll
        for (int by = 1; by < 32; by <<= 1) {
            const Sums o = {__shfl_up_sync(0xffffffffu, s.tiles, by), __shfl_up_sync(0xffffffffu, s.rows, by),
                            __shfl_up_sync(0xffffffffu, s.pieces, by), __shfl_up_sync(0xffffffffu, s.shorts, by),
                            __shfl_up_sync(0xffffffffu, s.wides, by)};
            if ((int)(threadIdx.x & 31) >= by)
                s.add(o);
        }
        return s;
    }
    __device__ __forceinline__ Sums of_lane(int lane) const
    {
        return {__shfl_sync(0xffffffffu, tiles, lane), __shfl_sync(0xffffffffu, rows, lane),
                __shfl_sync(0xffffffffu, pieces, lane), __shfl_sync(0xffffffffu, shorts, lane),
                __shfl_sync(0xffffffffu, wides, lane)};
    }
};

// One CTA, a few microseconds of latencies one after the other: everything
// between the loads and the stores stays in shared memory for up to kPlanEntries
// entries, warps without entries pass the barriers only, and the code is kept
// short, since each call runs it once, from cold.
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const __grid_constant__ bdla_cache c, const int32_t *cu_groups, const int32_t *shared,
            const __grid_constant__ Sizes z, const __grid_constant__ Plan p, DeviceStatus *st)
{
    extern __shared__ int smem_ints[];
    __shared__ int64_t s_positions;
    __shared__ int s_tiles, s_pieces[kSizes], s_longest;
    __shared__ Sums of_warp[32];
    next_may_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int NG = z.n_groups, B = z.B, E = NG + B;
    int *base = E <= kPlanEntries ? smem_ints : p.scratch;
    int *cu = base, *most = cu + NG + 1, *len = most + NG, *group = len + E;   // most: before the short ones are dropped
    const int cap = c.max_pages * c.page;

    // groups: inside the batch and in order, or there are none
    const int first_len = tid < B ? c.lens[tid] : 0;
    bool bad = false;
    for (int g = tid; g <= NG; g += kPlanThreads) {
        const int n0 = cu_groups[g];
        cu[g] = n0;
        if (g == NG)
            break;
        const int n1 = cu_groups[g + 1], s = shared[g];
        bad |= n0 < 0 || n1 < n0 || n1 > B;
        if (s < 0)
            set_status(st, BDLA_ERR_DEVICE, (unsigned)g);
        most[g] = min(max(s, 0), cap);
    }
    if (tid < kSizes)
        s_pieces[tid] = 0;
    if (tid < 32)
        of_warp[tid] = {};
    if (tid == 0) {
        s_tiles = s_longest = 0;
        s_positions = 0;
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0)
        set_status(st, BDLA_ERR_DEVICE, 0u);
    // a group shares what the shortest of its sequences has in the cache
    for (int b = tid; b < B; b += kPlanThreads) {
        const int l = b == tid ? first_len : c.lens[b];
        int g = -1;
        if (!bad) {
            int lo = 0, hi = NG;   // the last offset at or before b
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= b)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            g = lo < NG && cu[lo] <= b ? lo : -1;
        }
        if (g >= 0)
            atomicMin(&most[g], max(l, 0));
        group[b] = g;
        p.group[b] = g;
        // what the sequence has all in all
        const int64_t all = (int64_t)l + z.T;
        if (l < 0 || all > cap)
            set_status(st, BDLA_ERR_DEVICE, (unsigned)b);
        len[NG + b] = l < 0 ? 0 : (int)(all < cap ? all : cap);
    }
    __syncthreads();
    // one sequence reads nothing twice, and a short prefix is not worth the joining
    const int rows_of = z.T * z.G;
    const auto taken = [&](int g) {
        if (g < 0 || bad)
            return 0;
        const int n = cu[g + 1] - cu[g];
        const int64_t saved = (int64_t)(n - 1) * most[g] * z.Hk * z.D * 2;
        return n < 2 || saved < (z.wide && n * rows_of > kNarrowRows ? z.least_wide : z.least_narrow) ? 0 : most[g];
    };
    const int mr_log = z.narrow_tiles == 1 ? 4 : 5;
    const auto rows = [&](int e, int n) { return e >= NG ? rows_of : n > 0 ? (cu[e + 1] - cu[e]) * rows_of : 0; };
    const auto wide = [&](int e, int R) { return e >= NG ? z.own_wide : z.wide && R > kNarrowRows; };
    // blocks of two row tiles and of one, and their line
    const auto full = [](int R) { return (R + BT - 1) / kWideTile; };
    const auto single = [](int R) { return (R + BT - 1) / BT & 1; };
    const auto line_of = [&](int R, int nt) { return nt > 0 ? z.Hk * (full(R) * (2 * nt + kRun) + single(R) * (nt + kRun)) : 0; };
    const auto blocks = [&](int R) { return (R + (1 << mr_log) - 1) >> mr_log; };
    int tiles = 0;
    int64_t positions = 0;
    for (int e = tid; e < E; e += kPlanThreads) {
        const int n = e < NG ? taken(e) : len[e] - taken(group[e - NG]), R = rows(e, n);
        len[e] = n;
        if (wide(e, R))
            tiles += line_of(R, tiles_of(n));
        else
            positions += (int64_t)blocks(R) * n;
    }
    if (warp * 32 < E) {
        tiles = __reduce_add_sync(0xffffffffu, tiles);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1)
            positions += __shfl_xor_sync(0xffffffffu, positions, w);
        if (lane == 0) {
            atomicAdd(&s_tiles, tiles);
            atomicAdd(reinterpret_cast<unsigned long long *>(&s_positions), (unsigned long long)positions);
        }
    }
    __syncthreads();
    tiles = s_tiles;
    positions = s_positions;
    const int per_cta = max(kLeastLine, over(tiles, z.ctas));

    // The narrow pieces' size: their work (a piece costs its start-up, about 128
    // positions) spread over the CTAs that the GPU holds, plus the last piece's
    // own length, plus what the join reads of the longest entry's pieces.  At
    // least the size that keeps the list inside its bounds.
    const int64_t least64 = z.most > 0 ? (positions + z.extra - 1) / z.extra : 0;
    int size = least64 > INT32_MAX - 128 ? INT32_MAX - 127 : ((int)least64 + 63) / 64 * 64;
    if (z.most > 0 && size <= 128 << (kSizes - 1)) {
        for (int e0 = warp * 32; e0 < E; e0 += kPlanThreads) {
            const int e = e0 + lane, n = e < E ? len[e] : 0, R = e < E ? rows(e, n) : 0;
            const bool mine = e < E && !wide(e, R);
            const int x = mine ? blocks(R) : 0, some = mine && e >= NG ? 1 : 0;
            const int longest = __reduce_max_sync(0xffffffffu, mine ? n : 0);
            int sum = 0;
#pragma unroll
            for (int i = 0; i < kSizes; ++i) {
                const int all = __reduce_add_sync(0xffffffffu, max(x * ((n + (128 << i) - 1) >> (7 + i)), some));
                sum = lane == i ? all : sum;
            }
            if (lane < kSizes)
                atomicAdd(&s_pieces[lane], sum);
            if (lane == kSizes)
                atomicMax(&s_longest, longest);
        }
        __syncthreads();
        // one size a lane, the cheapest to all
        const int i = lane % kSizes;
        float cost = 128 << i < size ? INFINITY
                                     : ((float)positions + 128.0f * (float)s_pieces[i]) * z.heads_per_slot + (float)(128 << i) +
                                           4.0f * (float)((s_longest + (128 << i) - 1) >> (7 + i));
        size = 128 << i;
#pragma unroll
        for (int w = 1; w < kSizes; w <<= 1) {
            const float c2 = __shfl_xor_sync(0xffffffffu, cost, w);
            const int s2 = __shfl_xor_sync(0xffffffffu, size, w);
            if (c2 < cost || (c2 == cost && s2 < size)) {
                cost = c2;
                size = s2;
            }
        }
    }
    size = max(size, 64);   // (no narrow piece: not looked at)

    // places of everything, entries in order
    Sums done = {};
    for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
        const int e = e0 + tid;
        Sums m = {};
        int n = 0, R = 0, nb = 0, np = 0, nt = 0, first = 0;
        bool direct = false;   // not even a group's sums are joined to one piece
        if (e < E) {
            n = len[e];
            R = rows(e, n);
            const bool w = wide(e, R);
            nb = w ? 0 : blocks(R);
            first = e < NG ? 0 : taken(group[e - NG]);
            if (w) {
                nt = tiles_of(n);
                m.tiles = line_of(R, nt);
                m.rows = nt > 0 ? (over(full(R) > 0 ? 2 * nt : nt, per_cta) + 1) * R * z.Hk : 0;
                m.wides = nt > 0 ? (full(R) > 0) + single(R) : 0;
            } else {
                np = n > 0 ? over(n, size) : e >= NG;
                direct = first == 0 && np == 1 && e >= NG;
                const bool shorter = n - (np - 1) * size < size / 2;   // the last piece: the others are whole
                m.pieces = nb * (np - shorter);
                m.shorts = nb * shorter;
                m.rows = direct ? 0 : np * R * z.Hk;
            }
        }
        const bool active = e0 + warp * 32 < E;
        const Sums upto = active ? m.scanned() : m;
        if (e0 > 0)
            __syncthreads();   // the sums of the chunk before have been read
        if (lane == 31)
            of_warp[warp] = upto;
        __syncthreads();
        if (!active)
            continue;   // (in the last chunk; `done` is read by warp 0, which always has entries)
        const Sums warps = of_warp[lane].scanned(), before = warps.of_lane(max(warp - 1, 0));
        Sums at = done;
        if (warp > 0)
            at.add(before);
        done.add(warps.of_lane(31));
        at.tiles += upto.tiles - m.tiles;
        at.rows += upto.rows - m.rows;
        at.pieces += upto.pieces - m.pieces;
        at.shorts += upto.shorts - m.shorts;
        at.wides += upto.wides - m.wides;
        // A lane writes what its entry has few of, the warp together where there are many: the pieces of the narrow
        // list, and the CTAs whose first tile lies in the entry.
        int w0 = 0, w1 = 0, w2 = 0;   // CTAs from w0 on begin in the entry's blocks of two row tiles, from w1 on in the last
        Work piece = {};
        if (e < E) {
            const int b = e >= NG ? e - NG : n > 0 ? cu[e] : 0, base1 = at.tiles + z.Hk * full(R) * (2 * nt + kRun);
            piece = {b, first, n, e < NG ? kSeen : max(c.lens[b], 0), b * z.T, R, nb, direct ? -1 : at.rows};
            p.parts[e] = {at.tiles, nt, R, at.rows, direct ? -1 : np, piece.tok0, base1, full(R)};
            if (nt > 0) {
                WideEntry x = {at.tiles, b, piece.tok0, R, first, first + n, piece.len, nt, at.rows, 0, full(R), 2};
                WideEntry *to = p.wide + at.wides;
                if (full(R) > 0)
                    *to++ = x;
                x.base = base1;
                x.rb0 = full(R);
                x.rb1 = x.rb0 + 1;
                x.row_tiles = 1;
                if (single(R))
                    *to = x;
                w0 = over(at.tiles, per_cta);
                w1 = over(base1, per_cta);
                w2 = over(at.tiles + m.tiles, per_cta);
            }
        }
        const int second = at.wides + (full(R) > 0);   // the entry of one row tile
        // piece i of `pieces` (x: k1 positions, row0 blocks of rows), u0 long and s0 short ones before the entry's
        const auto write = [&](const Work &x, int pieces, int i, int u0, int s0) {
            const int n = min(x.k1 - i * size, size), last = i + 1 == pieces && n < size / 2;
            for (int rb = 0; rb < x.row0; ++rb)
                p.list[last ? z.most - 1 - (s0 + rb) : u0 + i * x.row0 + rb] =
                    {x.b, x.k0 + i * size, x.k0 + i * size + n, x.len, x.tok0, x.R, rb << mr_log,
                     x.part < 0 ? -1 : x.part + i * z.Hk * x.R};
        };
        if (np <= kFew)
            for (int i = 0; i < np; ++i)
                write(piece, np, i, at.pieces, at.shorts);
        if (w2 - w0 <= kFew)
            for (int w = w0; w < w2; ++w)
                p.first_entry[w] = w < w1 ? at.wides : second;
        for (uint32_t left = __ballot_sync(0xffffffffu, np > kFew || w2 - w0 > kFew); left != 0; left &= left - 1) {
            const int l = __ffs(left) - 1;
            const auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, l); };
            const int pieces = of(np), to = of(w2), turn = of(w1), from = of(w0), which = of(at.wides), then = of(second), u0 = of(at.pieces), s0 = of(at.shorts);
            const Work x = {of(piece.b), of(piece.k0), of(piece.k1), of(piece.len), of(piece.tok0), of(piece.R), of(piece.row0),
                            of(piece.part)};
            if (pieces > kFew)
                for (int i = lane; i < pieces; i += 32)
                    write(x, pieces, i, u0, s0);
            for (int w = from + lane; w < to; w += 32)
                p.first_entry[w] = w < turn ? which : then;
        }
    }
    if (tid == 0)
        *p.head = {tiles, per_cta, {done.pieces, z.most - done.shorts}};
}

// ---------------------------------------------------------------- wide
constexpr int kFetchWarps = 3;
constexpr int kThreads = 32 + 32 * kFetchWarps + 256;

// One CTA's way through its share of all tiles: runs of consecutive tiles of one
// (entry, block of rows, key head).  Every warp walks it by itself, in shared
// memory: it is looked at between runs, and its registers are wanted within them.
struct Walk {
    WideEntry en;
    const WideEntry *at;
    int rb, kh, t0, n, piece, from, end;   // from: of the run's tile 0 on the line; end: of the CTA's part of it
    __device__ __forceinline__ void settle()
    {
        const int x = from + t0 * en.row_tiles;
        n = x < end ? min(en.nt - t0, (end - x + en.row_tiles - 1) / en.row_tiles) : 0;
    }
    __device__ __forceinline__ void step(int Hk)
    {
        from += en.nt * en.row_tiles + kRun;
        t0 = piece = n = 0;
        if (from >= end)
            return;
        if (++kh == Hk) {
            kh = 0;
            if (++rb == en.rb1) {
                en = *++at;
                rb = en.rb0;
            }
        }
        settle();
    }
    // One lane.  n = 0: there is no tile.
    __device__ __forceinline__ void begin(const Plan &p, int Hk, int cta)
    {
        const Head h = *p.head;
        const int which = p.first_entry[cta], x = cta * h.per_cta;   // (which: if there is a line to walk)
        end = min(h.line, x + h.per_cta);
        n = 0;
        if (x >= h.line)
            return;
        at = p.wide + which;
        en = *at;
        const int whole = en.nt * en.row_tiles + kRun, unit = (x - en.base) / whole;
        from = en.base + unit * whole + kRun;
        t0 = x > from ? (x - from + en.row_tiles - 1) / en.row_tiles : 0;   // the first tile that starts at x or behind
        rb = unit / Hk;
        kh = unit - rb * Hk;
        rb += en.rb0;
        piece = cta - from / h.per_cta;
        settle();
        if (n == 0)   // the last tile began before x
            step(Hk);
    }
    // The next run, by the whole warp; false: there is none.
    __device__ __forceinline__ bool next(int Hk)
    {
        __syncwarp();   // all have looked at the run before
        if ((threadIdx.x & 31) == 0)
            step(Hk);
        __syncwarp();
        return n > 0;
    }
    __device__ __forceinline__ int row_tiles() const { return en.row_tiles; }
};

template <int D> struct WideSmem {
    static constexpr int kPanels = D / 64;
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kStages = D == 128 ? 5 : 8;
    // `valid` of a tile is written again by the tile eight later, which is looked up when at most six tiles (the ring
    // and the warps' own) lie between it and the softmax.
    static constexpr int kSlots = 8;
    alignas(1024) unsigned char q[2][kTile];
    alignas(1024) unsigned char ring[kStages][kTile];   // K_0 V_0 K_1 V_1 ...
    int row[kFetchWarps][BT];    // cache row of the positions of a warp's tile, -1: not seen
    uint32_t valid[kSlots][4];   // positions of a tile that may be seen
    uint64_t full[kStages], empty[kStages], q_full[2], s_full[2], o_done[2], merge, merged, drain, never;
    uint64_t p_ready[2][2];   // weights of the first and of the last 64 positions of a tile
    uint64_t wait_ns;
    Walk walk[1 + kFetchWarps + 8];   // of each warp
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(WideSmem<128>) <= kMaxSmem && sizeof(WideSmem<64>) <= kMaxSmem, "shared memory of a CTA");

// The pipeline of the wide kernel of bdla_cache_wide.cu, kept running from one
// run of tiles to the next: tiles, ring stages and barrier phases count on, keys
// and values of the next run are fetched while the last of this one is worked
// on, and only the rows (queries in, sums out) change hands.  All CTAs get the
// same length of the line, on which tiles and changes of rows are weighed.  Where a block has 128 rows or fewer there is no second
// row tile to turn to: both softmax groups then take the same rows and every
// second tile of positions, and the first reads the output of both out of tensor
// memory at the run's end.  `run` as there.
// DRAFTS: there are entries with new tokens among their positions (the sequences' own).
template <int D, bool DRAFTS>
__global__ void __launch_bounds__(kThreads, 1)
shared_wide_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, int run,
                   const __grid_constant__ Call a, const __grid_constant__ Plan plan, uint64_t wait_ns, int stall)
{
    using Smem = WideSmem<D>;
    constexpr int NS = Smem::kStages, SL = Smem::kSlots, NP = Smem::kPanels, kChunks = D / 8;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bdla_cache &c = a.c;
    const int T = a.T, Hq = a.Hq, Hk = a.Hk, G = Hq / Hk;
    next_may_start();
    if ((smem_u32(smem_raw) & 1023u) != 0u) {
        if (tid == 0)
            set_status(a.st, BDLA_ERR_DEVICE, 0xA11u);
        wait_for_previous();
        return;
    }
    if (warp == 0) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    } else if (tid == 32) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sm.full[s], 32);
            mbar_init(&sm.empty[s], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sm.q_full[x], BT);
            mbar_init(&sm.s_full[x], 1);
            mbar_init(&sm.p_ready[x][0], BT);
            mbar_init(&sm.p_ready[x][1], BT);
            mbar_init(&sm.o_done[x], 1);
        }
        mbar_init(&sm.merge, BT);
        mbar_init(&sm.merged, BT);
        mbar_init(&sm.drain, 1);
        mbar_init(&sm.never, 1);
        sm.abort_flag = 0;
        sm.wait_ns = wait_ns;
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_for_previous();   // the plan is there
    const uint32_t tmem = sm.tmem_base;
    volatile int *abort_flag = &sm.abort_flag;
    Walk &walk = sm.walk[warp];
    if (lane == 0)
        walk.begin(plan, Hk, blockIdx.x);
    __syncwarp();
    const bool any = walk.n > 0;
    const int stall_at = walk.n > 1 ? 1 : 0;   // test hook: the tile at which a role stalls

    if (warp == 0) {
        // ---------------------------------------------------------------- MMA issuer
        const uint64_t q[2] = {rows_desc(smem_u32(sm.q[0])), rows_desc(smem_u32(sm.q[1]))};
        bool ok = any;
        int j0 = 0;              // tiles before this run
        int runs[2] = {0, 0};    // runs before this one that a softmax group has had tiles of
        int had[2] = {0, 0};     // and its tiles
        while (ok) {
            // a tile's two turns, one for each row tile; or two tiles' turns, one for each group
            const int n = walk.n, turns = walk.row_tiles() == 1, step = turns ? 2 : 1;
            auto issue_qk = [&](int w, int j) {
                const int it = 2 * j;
                if (!warp_wait(&sm.full[it % NS], (it / NS) & 1, &sm.wait_ns, abort_flag))
                    return false;
                tc_fence_after();
                const uint64_t k = rows_desc(smem_u32(sm.ring[it % NS]));
                if (elect_one()) {
                    mma_rows<D>(tmem + BT * w, q[w], k);
                    umma_commit(&sm.s_full[w]);
                    if (turns || w == 1)   // the last reader of this key tile
                        umma_commit(&sm.empty[it % NS]);
                }
                __syncwarp();
                return true;
            };
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int x = turns ? w : 0;
                if (!ok || x >= n)
                    continue;
                ok = warp_wait(&sm.q_full[w], (uint32_t)(runs[w]++ & 1), &sm.wait_ns, abort_flag);
                tc_fence_after();
                ok = ok && issue_qk(w, j0 + x);
            }
            for (int x0 = 0; ok && x0 < n; x0 += step) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int x = turns ? x0 + w : x0;
                    if (!ok || x >= n)
                        continue;
                    const int it = 2 * (j0 + x) + 1;
                    const uint32_t phase = (uint32_t)(had[w] & 1);
                    ++had[w];
                    const bool hook = stall == BDLA_STALL_MMA && j0 + x == stall_at;
                    ok = warp_wait(&sm.full[it % NS], (it / NS) & 1, &sm.wait_ns, abort_flag) &&
                         warp_wait(hook ? &sm.never : &sm.p_ready[w][0], hook ? 0u : phase, &sm.wait_ns, abort_flag);
                    if (!ok)
                        continue;
                    tc_fence_after();
                    const uint64_t v = sum_desc(smem_u32(sm.ring[it % NS]));
                    const uint32_t acc = tmem + 2 * BT + BT * w, wt = tmem + BT * w;
                    if (elect_one())
                        mma_sum<D, 32, 0, BT / 32>(acc, wt, v, x0 > 0);
                    __syncwarp();
                    ok = warp_wait(&sm.p_ready[w][1], phase, &sm.wait_ns, abort_flag);
                    if (!ok)
                        continue;
                    tc_fence_after();
                    if (elect_one()) {
                        mma_sum<D, 32, BT / 32, BT / 16>(acc, wt, v, true);
                        if (turns || w == 1)
                            umma_commit(&sm.empty[it % NS]);
                        if (x + step >= n)
                            umma_commit(&sm.o_done[w]);
                    }
                    __syncwarp();
                    if (x + step < n)
                        ok = issue_qk(w, j0 + x + step);
                }
            }
            j0 += n;
            if (!walk.next(Hk))
                break;
        }
        if (any && !ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(a.st, BDLA_ERR_TIMEOUT, 0x40u);
        }
        // every MMA issued above has completed before TMEM is released
        if (elect_one())
            umma_commit(&sm.drain);
        __syncwarp();
        mbar_wait(&sm.drain, 0, kDrainNs);
    } else if (warp < 4) {
        // ---------------------------------------------------------------- fetching
        const int fw = warp - 1;
        bool ok = true;
        int issued = -1;   // this warp's last tile asked of TMA
        int j1 = walk.n;   // tiles up to the end of this run
        // a tile of this warp: its first position, where they end and which are committed, its heads and table
        struct Tile {
            int t, end, len, kh, b;
        };
        const auto tile_at = [&](int j, Tile &x) {   // j does not go back; false: there is none
            while (j >= j1) {
                if (!walk.next(Hk))
                    return false;
                j1 += walk.n;
            }
            x = {walk.en.first + (walk.t0 + j - (j1 - walk.n)) * BT, walk.en.end, walk.en.len, walk.kh, walk.en.b};
            return true;
        };
        const auto lookup = [&](const Tile &x, int (&pg)[4]) {
            const int32_t *table = c.pages + (int64_t)x.b * c.max_pages;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int t = x.t + 4 * lane + u;
                pg[u] = t < x.end ? table[a.div.entry(t)] : -1;
            }
        };
        Tile now{}, ahead{};
        int pg[4];
        bool more = any && tile_at(fw, ahead);
        if (more)
            lookup(ahead, pg);
        for (int j = fw; ok && more; j += kFetchWarps) {
            now = ahead;
            const uint64_t seen = DRAFTS && now.t + BT > now.len ? sees_any(a.tree, now.b, T, lane) : 0;
            int row[4];
            uint32_t bits = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int t = now.t + 4 * lane + u;
                bool live = t < now.end && (!DRAFTS || t < now.len || ((seen >> (t - now.len)) & 1));
                if (live && (pg[u] < 0 || pg[u] >= c.n_pages)) {
                    set_status(a.st, BDLA_ERR_DEVICE, (unsigned)now.b);
                    live = false;
                }
                row[u] = live ? pg[u] * c.page + a.div.offset(t) : -1;
                bits |= (live ? 1u : 0u) << u;
            }
            const bool whole = run > 0 && now.t % run == 0 && __all_sync(0xffffffffu, bits == 15u);
            bits <<= 4 * (lane & 7);
#pragma unroll
            for (int x = 1; x < 8; x <<= 1)
                bits |= __shfl_xor_sync(0xffffffffu, bits, x);
            if ((lane & 7) == 0)
                sm.valid[j % SL][lane >> 3] = bits;
            if (!whole) {
                *reinterpret_cast<int4 *>(&sm.row[fw][4 * lane]) = make_int4(row[0], row[1], row[2], row[3]);
                __syncwarp();
            }
            more = tile_at(j + kFetchWarps, ahead);
            if (more)
                lookup(ahead, pg);
#pragma unroll 1
            for (int v = 0; ok && v < 2; ++v) {
                const int it = 2 * j + v, s = it % NS;
                const bool hook = stall == BDLA_STALL_PRODUCER && it == 2 * stall_at;
                if (it >= NS || hook)
                    ok = warp_wait(hook ? &sm.never : &sm.empty[s], hook ? 0u : (uint32_t)((it / NS - 1) & 1), &sm.wait_ns,
                                   abort_flag);
                if (!ok)
                    break;
                if (whole) {
                    if (elect_one())
                        mbar_arrive_expect_tx(&sm.full[s], (uint32_t)Smem::kTile);
                    else
                        mbar_arrive(&sm.full[s]);
                    __syncwarp();
                    for (int x = 0; x < BT; x += run) {
                        const int first = __shfl_sync(0xffffffffu, row[0], x >> 2);
                        if (elect_one()) {
#pragma unroll
                            for (int p = 0; p < NP; ++p)
                                tma_load_2d(sm.ring[s] + p * kPanel + x * 128, v ? &tv : &tk, &sm.full[s], now.kh * D + 64 * p,
                                            first);
                        }
                        __syncwarp();
                    }
                    issued = it;
                } else {
                    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(v ? c.v : c.k) + (int64_t)now.kh * D;
                    const int ch = lane % kChunks;
                    const uint32_t dst = smem_u32(sm.ring[s]) + (ch >> 3) * kPanel;
#pragma unroll 8
                    for (int x = lane / kChunks; x < BT; x += 32 / kChunks) {
                        const int at_row = sm.row[fw][x];
                        cp16(dst + sw128_offset(x, ch & 7), src + (int64_t)max(at_row, 0) * Hk * D + 8 * ch, at_row >= 0);
                    }
                    cp_commit();
                    if (v == 1) {   // keys first, while the values are on their way
                        cp_wait<1>();
                        fence_proxy_async_smem();
                        mbar_arrive(&sm.full[(it - 1) % NS]);
                        cp_wait<0>();
                        fence_proxy_async_smem();
                        mbar_arrive(&sm.full[s]);
                    }
                }
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(a.st, BDLA_ERR_TIMEOUT, 0x41u);
            // this warp's copies in flight land before the CTA exits
            cp_wait<0>();
            for (int it = max(issued - NS + 1, 0); it <= issued; ++it)
                if ((it >> 1) % kFetchWarps == fw)
                    mbar_wait(&sm.full[it % NS], (it / NS) & 1, kDrainNs);
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const int w = warp >= 8, q4 = warp & 3, r = 32 * q4 + lane;
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const uint32_t t_s = tmem + BT * w + lane_off, t_o = tmem + 2 * BT + BT * w + lane_off;
        const float cs = a.scale * kLog2e;
        bool ok = any;
        float2 *second = reinterpret_cast<float2 *>(sm.q[1]);   // group 1's maxima and sums (its queries are read by then)
        int j0 = 0, had = 0, runs = 0, merges = 0;   // tiles before this run; tiles, runs and shared runs of this group
        while (ok) {
            const int n = walk.n, turns = walk.row_tiles() == 1;
            if (turns && w >= n) {   // one tile, which is the other group's
                j0 += n;
                if (!walk.next(Hk))
                    break;
                continue;
            }
            int i;   // the row's token
            {
                // the warp's 32 rows, whole rows at a time
                const int rr = walk.rb * kWideTile + (turns ? 0 : w * BT) + r, R = walk.en.R;
                i = rr < R ? rr / G : 0;
                const int mine = rr < R ? (walk.en.tok0 + i) * Hq + walk.kh * G + rr - i * G : -1;
                const int ch = lane % kChunks;
#pragma unroll 8
                for (int x = 0; x < kChunks; ++x) {
                    const int y = x * (32 / kChunks) + lane / kChunks, row = __shfl_sync(0xffffffffu, mine, y);
                    *reinterpret_cast<uint4 *>(sm.q[w] + (ch >> 3) * kPanel + sw128_offset(32 * q4 + y, ch & 7)) =
                        row >= 0 ? reinterpret_cast<const uint4 *>(a.q + (int64_t)row * D)[ch] : make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                tc_fence_before();   // the sums of the run before have been read
                mbar_arrive(&sm.q_full[w]);
            }
            const int len = DRAFTS ? walk.en.len : kSeen, step = turns ? 2 : 1, x0 = turns ? w : 0;
            const uint64_t see = DRAFTS && walk.en.end > len ? sees(a.tree, walk.en.b, T, i) : 0;
            RowSoftmax row;
            int t0 = walk.en.first + (walk.t0 + x0) * BT;
            for (int x = x0; x < n; x += step, t0 += step * BT) {
                const int j = j0 + x;
                const bool hook = stall == BDLA_STALL_EPILOGUE && j == stall_at;
                ok = warp_wait(hook ? &sm.never : &sm.s_full[w], hook ? 0u : (uint32_t)(had & 1), &sm.wait_ns, abort_flag);
                ++had;
                if (!ok)
                    break;
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tmem_ld32(t_s + 32 * k, s[k]);
                tmem_ld_wait();
                uint32_t all = 0xffffffffu;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    all &= sm.valid[j % SL][k];
                if (all != 0xffffffffu || (DRAFTS && t0 + BT > len)) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // what this row sees of the 32 positions: the context, and its bits of the new tokens
                        const int p0 = t0 + 32 * k - len;   // first of them as a new token
                        uint32_t mask = p0 <= -32 ? 0xffffffffu
                                                  : p0 < 0 ? ((1u << -p0) - 1) | (uint32_t)(see << -p0)
                                                           : p0 < 64 ? (uint32_t)(see >> p0) : 0u;
                        mask = (DRAFTS ? mask : 0xffffffffu) & sm.valid[j % SL][k];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            s[k][e] = (mask >> e) & 1 ? s[k][e] : 0xff800000u;
                    }
                }
                row_weights<D>(s, cs, t_s, t_o, x == x0, row, [&](int half) { mbar_arrive(&sm.p_ready[w][half]); });
            }
            if (ok)
                ok = warp_wait(&sm.o_done[w], (uint32_t)(runs++ & 1), &sm.wait_ns, abort_flag);
            if (!ok)
                break;
            tc_fence_after();
            j0 += n;
            float f0 = 1.0f, f1 = 0.0f;   // factors of this group's sums and of the other's
            const bool both = turns && n > 1;
            if (both) {
                // the same rows: group 1 hands its maximum and sum over, and group 0 reads the output of both
                if (w == 1) {
                    second[r] = make_float2(row.m, row.l);
                    tc_fence_before();
                    mbar_arrive(&sm.merge);
                    ok = warp_wait(&sm.merged, (uint32_t)(merges++ & 1), &sm.wait_ns, abort_flag);
                    if (!ok || !walk.next(Hk))
                        break;
                    continue;
                }
                ok = warp_wait(&sm.merge, (uint32_t)(merges++ & 1), &sm.wait_ns, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                const float2 o = second[r];
                const float m = fmaxf(row.m, o.x);
                f0 = row.m == m ? 1.0f : ex2((row.m - m) * cs);
                f1 = o.x == m ? 1.0f : ex2((o.x - m) * cs);
                row.m = m;
                row.l = fmaf(row.l, f0, o.y * f1);
            }
            const int R = walk.en.R, rr = walk.rb * kWideTile + (turns ? 0 : w * BT) + r;
            const int64_t pt = (int64_t)walk.en.part + ((int64_t)walk.piece * Hk + walk.kh) * R + rr;
            // 32 rows of 128 bytes at a time through the warp's own rows of its query tile (read by now), so that whole
            // lines leave
            uint4 *stage = reinterpret_cast<uint4 *>(sm.q[w] + q4 * 4096);
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
                uint32_t y[32];
                tmem_ld32(t_o + 32 * k, y);
                if (both) {
                    uint32_t y1[32];
                    tmem_ld32(t_o + BT + 32 * k, y1);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        y[e] = __float_as_uint(fmaf(__uint_as_float(y[e]), f0, __uint_as_float(y1[e]) * f1));
                } else {
                    tmem_ld_wait();
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    stage[lane * 8 + (e ^ (lane & 7))] = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int x = 4 * u + (lane >> 3);   // row of the warp
                    const uint4 z = stage[x * 8 + ((lane & 7) ^ (x & 7))];
                    if (rr - lane + x < R)
                        *reinterpret_cast<uint4 *>(a.part_o + (pt - lane + x) * D + 32 * k + 4 * (lane & 7)) = z;
                }
                __syncwarp();
            }
            if (both) {
                tc_fence_before();   // the other group's output has been read
                mbar_arrive(&sm.merged);
            }
            if (rr < R)
                *reinterpret_cast<float2 *>(a.part_ml + 2 * pt) = make_float2(row.m, row.l);
            if (!walk.next(Hk))
                break;
        }
        if (any && !ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(a.st, BDLA_ERR_TIMEOUT, 0x42u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- join
// The pieces of a row: the group's, then the sequence's own.  W warps a row, each
// taking every W-th piece with a maximum of its own; their sums are added in
// order.
template <int D, int W>
__global__ void __launch_bounds__(W < 4 ? 128 : 32 * W)
shared_join_kernel(const __grid_constant__ Call a, const __grid_constant__ Plan plan, int n_groups, int64_t rows)
{
    constexpr int E = D / 32, kRows = W < 4 ? 4 / W : 1;
    __shared__ float red_l[kRows][W], red_m[kRows][W];
    __shared__ __align__(16) float red_o[kRows][W][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp / W, w = warp % W;
    const int64_t at = (int64_t)blockIdx.x * kRows + mine;
    const int T = a.T, Hq = a.Hq, Hk = a.Hk, G = Hq / Hk;
    const bool any = at < rows;
    const int h = any ? (int)(at % Hq) : 0, i = any ? (int)(at / Hq % T) : 0, b = any ? (int)(at / Hq / T) : 0;
    const int kh = h / G;
    wait_for_previous();
    const Head head = *plan.head;
    const int g = plan.group[b];
    // first row of the pieces' sums, the step from piece to piece, and how many there are
    const auto pieces = [&](int e, int64_t &first, int64_t &step) {
        const Parts x = plan.parts[e];
        const int rr = (b * T + i - x.tok0) * G + h % G;
        first = (int64_t)x.part + (int64_t)kh * x.R + rr;
        step = (int64_t)Hk * x.R;
        if (x.nt == 0)
            return x.np;
        const int rb = rr / kWideTile, row_tiles = rb < x.full ? 2 : 1;
        const int begin = kRun + (rb < x.full ? x.base + (rb * Hk + kh) * (2 * x.nt + kRun) : x.base1 + kh * (x.nt + kRun));
        return (begin + (x.nt - 1) * row_tiles) / head.per_cta - begin / head.per_cta + 1;
    };
    int64_t f0 = 0, s0 = 0, f1 = 0, s1 = 0;
    const int n1 = pieces(n_groups + b, f1, s1);
    const int n0 = g >= 0 && any ? pieces(g, f0, s0) : 0;
    const bool live = any && n1 >= 0;   // else finished by its own CTA
    if (W > 1 && !live)
        return;   // the whole CTA
    const int n = live ? n0 + n1 : 0;
    const auto place = [&](int s) { return s < n0 ? f0 + s * s0 : f1 + (s - n0) * s1; };
    const float cs = a.scale * 1.4426950408889634f;
    // rounds of 32 pieces of each warp, a lane's own piece's maximum and sum; sums of rows eight at a time, asked for
    // before the maximum is known
    float m = -INFINITY, l = 0.0f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        v[e] = 0.0f;
    for (int s0_ = 0; s0_ < n; s0_ += 32 * W) {
        const int mine_s = s0_ + w + W * lane;
        const float2 ml = mine_s < n ? *reinterpret_cast<const float2 *>(a.part_ml + 2 * place(mine_s)) : make_float2(-INFINITY, 0.0f);
        float top = ml.x;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        top = fmaxf(top, m);
        const float old = m == top ? 1.0f : ex2((m - top) * cs);
        m = top;
        const float f = ml.x == top ? 1.0f : ex2((ml.x - top) * cs);
        l *= old;
#pragma unroll
        for (int e = 0; e < E; ++e)
            v[e] *= old;
        const int here = min(32, (n - s0_ - w + W - 1) / W);   // pieces of this warp
        for (int u0 = 0; u0 < here; u0 += 8) {
            float y[8][E];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float *src = a.part_o + place(s0_ + w + W * (u0 + u)) * D + E * lane;
                const bool some = u0 + u < here;
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 z = some ? *reinterpret_cast<const float2 *>(src + e) : make_float2(0.0f, 0.0f);
                    y[u][e] = z.x;
                    y[u][e + 1] = z.y;
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float fu = __shfl_sync(0xffffffffu, f, u0 + u), lu = __shfl_sync(0xffffffffu, ml.y, u0 + u);
                if (u0 + u >= here)
                    continue;
                l = fmaf(lu, fu, l);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    v[e] = fmaf(y[u][e], fu, v[e]);
            }
        }
    }
    if (W > 1) {   // the warps' sums to one maximum
        if (lane == 0)
            red_m[mine][w] = m;
        __syncthreads();
        float top = m;
        for (int x = 0; x < W; ++x)
            top = fmaxf(top, red_m[mine][x]);
        const float f = m == top ? 1.0f : ex2((m - top) * cs);
        m = top;
        l *= f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            v[e] *= f;
    }
    if (W > 1) {
        if (lane == 0)
            red_l[mine][w] = l;
#pragma unroll
        for (int e = 0; e < E; ++e)
            red_o[mine][w][E * lane + e] = v[e];
        __syncthreads();
        if (w != 0)
            return;
        for (int x = 1; x < W; ++x) {
            l += red_l[mine][x];
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] += red_o[mine][x][E * lane + e];
        }
    }
    if (!live)
        return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(a.o + at * D + E * lane + e) = pack_bf16(v[e] * inv, v[e + 1] * inv);
    if (lane == 0)
        a.lse[at] = l == 0.0f ? -INFINITY : fmaf(m, a.scale, logf(l));
}

template <int D, bool DRAFTS> cudaError_t wide_go(const Call &a, const Plan &p, const Sizes &z, cudaStream_t stream)
{
    const size_t smem = sizeof(WideSmem<D>);
    const cudaError_t err = cudaFuncSetAttribute(shared_wide_kernel<D, DRAFTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    CUtensorMap tk{}, tv{};
    int run = a.c.page & -a.c.page;   // the largest power of two in the page
    run = run > BT ? BT : run;
    const int64_t rows = (int64_t)a.c.n_pages * a.c.page, width = (int64_t)a.Hk * D;
    if (run < 16 || rows == 0)
        run = 0;
    else if (!make_rows_map(&tk, a.c.k, width, rows, run) || !make_rows_map(&tv, a.c.v, width, rows, run))
        return cudaErrorInvalidValue;
    return launch_second(shared_wide_kernel<D, DRAFTS>, (unsigned)z.ctas, kThreads, smem, stream, tk, tv, run, a, p, g_wait_ns.load(),
                         g_test_stall[BDLA_KERNEL_ATTN_SHARED].load());
}

template <int D> cudaError_t join_go(const Call &a, const Plan &p, const Sizes &z, int64_t rows, cudaStream_t stream)
{
    // few rows have many pieces, and leave the SMs idle with a warp each
    return rows <= 16 * (int64_t)z.ctas
               ? launch_second(shared_join_kernel<D, 4>, (unsigned)rows, 128, 0, stream, a, p, z.n_groups, rows)
               : launch_second(shared_join_kernel<D, 1>, (unsigned)((rows + 3) / 4), 128, 0, stream, a, p, z.n_groups, rows);
}

}  // namespace

size_t shared_bytes(const bdla_attn_dims &d, int n_groups, int64_t max_keys)
{
    Plan p;
    return carve(sizes_of(d, n_groups, max_keys), nullptr, &p);
}

// The line (with a CTA's worth beyond it) and rows of the partial sums are 32-bit.
bool shared_fits(const bdla_attn_dims &d, int n_groups, int64_t max_keys)
{
    const Sizes z = sizes_of(d, n_groups, max_keys);
    const int64_t R = (int64_t)d.T * z.G, groups = z.wide ? R * d.B / kWideTile + (n_groups < d.B / 2 ? n_groups : d.B / 2) : 0;
    const int64_t blocks = (groups + (z.own_wide ? (R + kWideTile - 1) / kWideTile * d.B : 0)) * d.Hk;
    return z.rows <= INT32_MAX && blocks <= INT32_MAX && blocks * (2 * (max_keys / BT + 1) + kRun) <= INT32_MAX / 2;
}

cudaError_t launch_attn_shared(const __nv_bfloat16 *q, const bdla_cache &c, const int32_t *cu_groups, const int32_t *shared,
                               int n_groups, const uint64_t *tree, float scale, __nv_bfloat16 *o, float *lse,
                               const bdla_attn_dims &d, void *scratch, DeviceStatus *st, cudaStream_t stream)
{
    const Sizes z = sizes_of(d, n_groups, (int64_t)c.max_pages * c.page);
    Plan p;
    carve(z, static_cast<char *>(scratch), &p);
    Call a;
    a.q = q;
    a.c = c;
    if ((int64_t)c.n_pages * c.page == 0)   // no rows: nothing is read, from an address that exists all the same
        a.c.k = a.c.v = const_cast<__nv_bfloat16 *>(q);
    a.tree = tree;
    a.scale = scale;
    a.o = o;
    a.lse = lse;
    a.part_o = p.part_o;
    a.part_ml = p.part_ml;
    a.T = d.T;
    a.Hq = d.Hq;
    a.Hk = d.Hk;
    a.div = PageDiv::of(c.page);
    a.pieces = {1, 1, 1};
    a.st = st;
    a.list = p.list;
    a.n_list = &p.head->list;
    KernelMark mark_(BDLA_KERNEL_ATTN_SHARED, stream);
    const int entries = n_groups + d.B;
    plan_kernel<<<1, kPlanThreads, entries <= kPlanEntries ? plan_ints(n_groups, d.B) * sizeof(int) : 0, stream>>>(c, cu_groups, shared, z, p, st);
    cudaError_t err = cudaGetLastError();
    if (err == cudaSuccess && z.wide)
        err = d.d == 64 ? (z.own_wide ? wide_go<64, true>(a, p, z, stream) : wide_go<64, false>(a, p, z, stream))
                        : (z.own_wide ? wide_go<128, true>(a, p, z, stream) : wide_go<128, false>(a, p, z, stream));
    if (err == cudaSuccess && z.most > 0)
        err = launch_cached_list(a, d.d, z.narrow_tiles, z.most, stream);
    if (err != cudaSuccess)
        return err;
    const int64_t rows = (int64_t)d.B * d.T * d.Hq;
    return d.d == 64 ? join_go<64>(a, p, z, rows, stream) : join_go<128>(a, p, z, rows, stream);
}

}  // namespace bdla
