// moe_attend.cuh -- what the two attention kernels (moe_kv_attend.cu: few query
// rows; moe_kv_attend_tc.cu: many) share: the split of the work over blocks,
// the bounded waits, the producer of cache pages and the joining of tiles cut
// between blocks.  Included inside namespace moe { namespace { ... } }, after
// moe_device.cuh and moe_layer_device.cuh.
//
// A tile is TR query rows (new tokens of one sequence x query heads of one kv
// head, token after token).  The units are the pages of all (sequence, kv head,
// tile) in a row; each block (one per SM) takes an equal run of them, so ragged
// lengths balance without knowing them on the host.  Beginning and ending a tile
// costs time too: COST units without pages stand at the head of each.  A tile cut
// by a run's end is joined by the last block that arrives at it, in block order:
// the same bits every run.
#pragma once

constexpr int kPage = MOE_KV_PAGE;
constexpr int kMaxStages = 12;

// What a block knows of every sequence.
struct Seqs {
    long long cum[MOE_KV_MAX_SEQS + 1];  // units before sequence b
    int per_head[MOE_KV_MAX_SEQS];       // units of one kv head
    int q0[MOE_KV_MAX_SEQS], n[MOE_KV_MAX_SEQS], len[MOE_KV_MAX_SEQS];
};

// Bounded wait; a block that gave up sets its abort flag and goes on without
// waiting, so that every warp still reaches the block's barriers.
__device__ __forceinline__ void wait_or_abort(uint64_t *bar, uint32_t parity, const AttendParams &p, int *abort_flag)
{
    uint64_t t0 = 0;  // (reading the timer takes long: not before many tries have failed)
#pragma unroll 1
    for (uint32_t it = 1; !mbar_test(bar, parity); ++it) {
        if ((it & 31u) != 0) continue;
        if (*reinterpret_cast<volatile int *>(abort_flag)) return;
        const uint64_t t = gtimer();
        if (t0 == 0) t0 = t;
        if (static_cast<long long>(t - t0) > p.timeout_ns) {
            atomicOr(p.c.ctrl + 2, kErrTimeout);
            *reinterpret_cast<volatile int *>(abort_flag) = 1;
            return;
        }
    }
}

// Tokens that row r of a sequence sees (r = new token * group + head).
__device__ __forceinline__ int row_sees(int len, int n, int G, int r) { return max(len - n + r / G + 1, 0); }

// The tokens of a page that a tree's token sees, a bit each: those before the tree, and of
// the tree's, from slot -base of the page on, those in way (its own way to the root).
__device__ __forceinline__ uint64_t tree_page(uint32_t way, int base)
{
    const uint64_t its = way;
    if (base >= 0) return base < kPage ? its >> base : 0ull;
    return base > -kPage ? its << -base | ((1ull << -base) - 1ull) : ~0ull;
}

// The token before new token i of a tree, -1: none; a parent that is not an earlier token counts as none.
__device__ __forceinline__ int tree_parent(const AttendParams &p, int q0, int i)
{
    const int up = __ldg(p.parent + q0 + i);
    if (up < i && up >= -1) return up;
    atomicOr(p.c.ctrl + 2, kErrBadIndex);
    return -1;
}

// The tokens of W pages from pg on that new token i of a tree sees, a bit each: those
// before the tree (the sequence's first `past`), those on the way from i to the root.  A
// parent is an earlier token, so the way back ends; one that is not counts as a
// root.  (The way is walked for each page that holds tokens of the tree: a few loads
// that hit L1, against masks of all tokens kept for one or two steps.)
template <int W>
__device__ __forceinline__ void tree_sees(const AttendParams &p, int q0, int past, int i, int pg, uint64_t (&w)[W])
{
    const int base = pg * kPage - past;  // the tree's token in slot 0 of page pg
#pragma unroll
    for (int x = 0; x < W; ++x) {
        const int b = base + x * kPage;
        w[x] = b >= 0 ? 0ull : (b <= -kPage ? ~0ull : (1ull << -b) - 1ull);
    }
    const int first = max(base, 0);
    while (i >= first) {
        const int d = i - base;
#pragma unroll
        for (int x = 0; x < W; ++x)
            if ((d >> 6) == x) w[x] |= 1ull << (d & 63);
        const int up = __ldg(p.parent + q0 + i);
        if (up >= i || up < -1) {
            atomicOr(p.c.ctrl + 2, kErrBadIndex);
            break;
        }
        i = up;
    }
}

// Units of row tile j: COST, and its pages, or one where its last row sees
// nothing (the tile's zeros still have to be written).
template <int COST>
__device__ __forceinline__ int tile_units(int len, int n, int G, int TR, int j)
{
    const int last = min((j + 1) * TR, n * G) - 1;
    return COST + max(1, (row_sees(len, n, G, last) + kPage - 1) / kPage);
}

// Fill in the sequences and their units; all threads of the block.
template <int COST, bool TREE>
__device__ __forceinline__ void plan_units(const AttendParams &p, Seqs &sq, int G, int TR)
{
    const KvParams &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    for (int b = tid; b < c.B; b += blockDim.x) {
        const int a0 = c.q_off[b], a1 = c.q_off[b + 1], l = c.kv_len[b];
        const int q0 = min(max(a0, 0), c.N), q1 = min(max(a1, q0), c.N);
        // out of range, or too long for a tree: nothing is seen
        const int len = l < 0 || l > c.max_pages * kPage || (TREE && q1 - q0 > MOE_KV_MAX_TREE) ? 0 : l;
        if (blockIdx.x == 0 && (q0 != a0 || q1 != a1 || len != l)) atomicOr(c.ctrl + 2, kErrBadIndex);
        sq.q0[b] = q0;
        sq.n[b] = q1 - q0;
        sq.len[b] = len;
        const int rows = (q1 - q0) * G;
        sq.per_head[b] = rows == 0 ? 0 : (rows <= TR ? tile_units<COST>(len, q1 - q0, G, TR, 0) : -1);
    }
    __syncthreads();
    for (int b = wid; b < c.B; b += blockDim.x >> 5) {  // sequences of several tiles: a warp each
        if (sq.per_head[b] >= 0) continue;
        const int n = sq.n[b], len = sq.len[b], tiles = (n * G + TR - 1) / TR;
        int sum = 0;
        for (int j = lane; j < tiles; j += 32) sum += tile_units<COST>(len, n, G, TR, j);
        sum = __reduce_add_sync(0xffffffffu, sum);
        __syncwarp();
        if (lane == 0) sq.per_head[b] = sum;
    }
    __syncthreads();
    if (wid == 0) {
        long long run = 0;
        for (int b0 = 0; b0 < c.B; b0 += 32) {
            const int b = b0 + lane;
            const long long mine = b < c.B ? static_cast<long long>(sq.per_head[b]) * c.kv_heads : 0;
            long long sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (b < c.B) sq.cum[b] = run + sum - mine;
            run += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) sq.cum[c.B] = run;
    }
    __syncthreads();
}

// A run of units of one tile.
struct Segment {
    int b, h, tile, p0, p1;   // pages [p0, p1) of the tile (p1 = 0: none of it, nothing to do)
    int pe;                   // p1, or where the sequence's pages end before it
    int pages;                // of the whole tile
    int units;                // of the run
    long long start;          // the tile's first unit with a page
    __device__ __forceinline__ bool whole() const { return p0 == 0 && p1 == pages; }
};

// The tile that unit u lies in, and the run of it up to unit end (the whole warp).
template <int COST>
__device__ __forceinline__ Segment locate(const Seqs &s, int B, int G, int TR, long long u, long long end)
{
    Segment g;
    int lo = 0, hi = B - 1;
    while (lo < hi) {  // the last b with cum[b] <= u (u is below cum[B])
        const int mid = (lo + hi + 1) >> 1;
        if (s.cum[mid] <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    g.b = lo;
    const int n = s.n[lo], len = s.len[lo];
    const int rel = static_cast<int>(u - s.cum[lo]);
    g.h = rel / s.per_head[lo];
    int r = rel - g.h * s.per_head[lo];
    const int tiles = (n * G + TR - 1) / TR;
    g.tile = 0;
    int units = tile_units<COST>(len, n, G, TR, 0);
    if (tiles > 1) {
        const int lane = threadIdx.x & 31;
        for (int j0 = 0; j0 < tiles; j0 += 32) {  // 32 tiles at a time (the whole warp)
            const int mine = j0 + lane < tiles ? tile_units<COST>(len, n, G, TR, j0 + lane) : 0;
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned m = __ballot_sync(0xffffffffu, sum > r);
            if (m) {
                const int l = __ffs(m) - 1;
                g.tile = j0 + l;
                units = __shfl_sync(0xffffffffu, mine, l);
                r -= __shfl_sync(0xffffffffu, sum, l) - units;
                break;
            }
            r -= __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    const int stop = static_cast<int>(min(static_cast<long long>(units), r + (end - u)));
    g.start = u - r + COST;
    g.pages = units - COST;
    g.units = stop - r;
    g.p0 = max(0, r - COST);
    g.p1 = max(0, stop - COST);
    g.pe = max(g.p0, min(g.p1, (len + kPage - 1) / kPage));
    return g;
}

// First unit of block c when U units are dealt out to G blocks.
__device__ __forceinline__ long long block_start(long long U, int G, int c)
{
    const long long q = U / G, r = U - q * G;
    return q * c + min(static_cast<long long>(c), r);
}
// The block whose run holds unit u.
__device__ __forceinline__ int block_of(long long U, int G, long long u)
{
    const long long q = U / G, r = U - q * G;
    const long long cut = (q + 1) * r;
    return static_cast<int>(u < cut ? u / (q + 1) : r + (u - cut) / q);
}

// Where a row's result goes.
__device__ __forceinline__ uint16_t *out_row(const AttendParams &p, int q0, int h, int G, int r)
{
    return p.o + (static_cast<size_t>(q0 + r / G) * p.c.q_heads + h * G + r % G) * p.c.D;
}
// 1 / (gain * l), 0 for a row that sees nothing (NaN stays).
__device__ __forceinline__ float inv_sum(float gain, float l) { return l > 0.f || l != l ? 1.f / (gain * l) : 0.f; }

// A block's partial result of a tile: slot 0 continues a tile, slot 1 starts
// one.  Maxima [TR], sums [TR], then the weighted sums [D / 4][TR][4], so that
// neighbouring rows are neighbours in memory.
__device__ __forceinline__ float *part_slot(const AttendParams &p, int block, bool starts)
{
    return p.part + (static_cast<size_t>(block) * 2 + (starts ? 1 : 0)) * attend_part_floats(p.c.D);
}

__device__ __forceinline__ float *part_at(float *part, int TR, int row, int d)
{
    return part + 2 * TR + ((d >> 2) * TR + row) * 4 + (d & 3);
}

// The output of R rows of a tile (of TR, the others are none of the sequence's) from the partial
// results of blocks c0 .. c1: a thread has one row and every (NT / R)-th group of four columns
// of it; the loads of A blocks go out together.  (What a block writes comes back at 64 bytes a
// cycle, the rate of an SM: 15 blocks' results of 64 rows of 128 take 8000 cycles with all
// threads at work, 16000 with the half that 128 rows would leave.)
template <int D, int NT, int TR, int R>
__device__ __forceinline__ void join_rows(const AttendParams &p, const Segment &s, int c0, int c1, int rows, int q0, int G, float gain,
                                          int tid)
{
    constexpr int IT = (R * (D / 4) + NT - 1) / NT, LOADS = TR == 128 ? 16 : 8, A = IT >= LOADS ? 1 : LOADS / IT;
    const int row = tid % R, g0 = tid / R, r = s.tile * TR + row;
    if (r >= rows || g0 >= D / 4) return;
    float M = -INFINITY, L = 0.f;
    float4 acc[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = c0; k0 <= c1; k0 += A) {
        float m[A], l[A];
        float4 v[A][IT];
#pragma unroll
        for (int x = 0; x < A; ++x) {
            float *q = part_slot(p, min(k0 + x, c1), min(k0 + x, c1) == c0);
            m[x] = k0 + x <= c1 ? __ldcg(q + row) : -INFINITY;
            l[x] = k0 + x <= c1 ? __ldcg(q + TR + row) : 0.f;
#pragma unroll
            for (int i = 0; i < IT; ++i)
                v[x][i] = __ldcg(reinterpret_cast<const float4 *>(part_at(q, TR, row, 4 * (g0 + i * (NT / R)))));
        }
#pragma unroll
        for (int x = 0; x < A; ++x) {
            const float mn = fmaxf(M, m[x]), ref = mn == -INFINITY ? 0.f : mn, f0 = ex2(M - ref), f1 = ex2(m[x] - ref);
            L = L * f0 + l[x] * f1;
            M = mn;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                acc[i].x = acc[i].x * f0 + v[x][i].x * f1;
                acc[i].y = acc[i].y * f0 + v[x][i].y * f1;
                acc[i].z = acc[i].z * f0 + v[x][i].z * f1;
                acc[i].w = acc[i].w * f0 + v[x][i].w * f1;
            }
        }
    }
    const float inv = inv_sum(gain, L);
    uint16_t *o = out_row(p, q0, s.h, G, r);
#pragma unroll
    for (int i = 0; i < IT; ++i)
        *reinterpret_cast<uint2 *>(o + 4 * (g0 + i * (NT / R))) =
            make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
}

// A tile cut between blocks: the last of them to arrive joins the partials of
// all and writes the output.  The block's NT consumers, this thread the tid-th of
// them, their partials written.
template <int D, int NT, int TR>
__device__ __forceinline__ void join_tile(const AttendParams &p, const Segment &s, long long U, int blocks, int rows, int q0,
                                          int G, float gain, int *last, int tid)
{
    const int c0 = block_of(U, blocks, s.start), c1 = block_of(U, blocks, s.start + s.pages - 1);
    __threadfence();
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
    if (tid == 0) {
        const uint32_t old = atom_add_acqrel_gpu(p.count + c0, 1u);
        *last = old == static_cast<uint32_t>(c1 - c0);
        if (*last) p.count[c0] = 0u;
    }
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
    if (!*last) return;
    __threadfence();
    const int left = rows - s.tile * TR;
    if (TR == 128 && left <= 32)
        join_rows<D, NT, TR, (TR < 32 ? TR : 32)>(p, s, c0, c1, rows, q0, G, gain, tid);
    else if (TR == 128 && left <= 64)
        join_rows<D, NT, TR, (TR < 64 ? TR : 64)>(p, s, c0, c1, rows, q0, G, gain, tid);
    else
        join_rows<D, NT, TR, TR>(p, s, c0, c1, rows, q0, G, gain, tid);
}

// 2^e * f covers a page's v scale: the exponent that the running maximum adds to
// a score, so that (weight x v scale) has its range whatever the scale.
__device__ __forceinline__ float scale_log2(float vs)
{
    const uint32_t u = __float_as_uint(vs);
    return static_cast<float>(max(-64, static_cast<int>(u >> 23) - 127 + ((u & 0x7FFFFFu) ? 1 : 0)));
}

// Ids and scales of up to 32 pages from pb on, a page a lane (id < 0: out of
// range, flagged).
struct PageInfo {
    int id;
    float ks, vs;
};
__device__ __forceinline__ PageInfo load_pages(const KvParams &c, const Segment &s, int pb)
{
    PageInfo r{-1, -1.f, 0.f};
    const int pg = pb + (threadIdx.x & 31);
    if (pg < s.pe) {
        const int id = c.pages[static_cast<size_t>(s.b) * c.max_pages + pg];
        if (id >= 0 && id < c.n_pages) {
            const size_t ph = static_cast<size_t>(id) * c.kv_heads + s.h;
            r = PageInfo{id, c.ks[ph], c.vs[ph]};
        } else {
            atomicOr(c.ctrl + 2, kErrBadIndex);
        }
    }
    return r;
}
