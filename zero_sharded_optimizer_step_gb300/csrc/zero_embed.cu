// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   y[i]       = scale * table[tok[i]]
//   dtable[r] (+)= scale * sum of dy[i] over the i with tok[i] = r, i ascending
//
// The sum of a table row is taken in fp32 in an order that depends on the
// tokens alone (positions in order within chunks of the sorted list, chunks in
// order), so that the same inputs give the same bits on every run: no float
// atomics anywhere.
#include "zero_elems.cuh"
#include "zero_ops.h"

namespace zgb {
namespace {

constexpr uint32_t kNone = 0xffffffffu;

// The table row token i names, or -1.
__device__ __forceinline__ int64_t token_row(const TokenArgs &t, int64_t i)
{
    const int64_t id = t.wide ? static_cast<const long long *>(t.ids)[i]
                              : (int64_t)static_cast<const int *>(t.ids)[i];
    return id == t.pad || id < 0 || id >= t.rows ? -1 : id;
}

// ------------------------------------------------------------- the lookup
//
// A warp copies up to 4 accesses a lane of one output row, all in flight at
// once; a wide row takes several warps.
constexpr int kEmbedFlight = 4;

template <int DT, int E>
__global__ void __launch_bounds__(kThreads)
embed_kernel(const __grid_constant__ EmbedArgs a, int segs)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t task = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t i = task / segs;
    const int seg = (int)(task - i * segs);
    if (i >= a.tok.n) return;
    const int64_t row = token_row(a.tok, i);
    if (row < 0 && a.bad && lane == 0 && seg == 0) {
        const int64_t id = a.tok.wide ? static_cast<const long long *>(a.tok.ids)[i]
                                      : (int64_t)static_cast<const int *>(a.tok.ids)[i];
        if (id != a.tok.pad) atomicAdd(a.bad, 1ull);
    }
    const int64_t c0 = ((int64_t)seg * kEmbedFlight * 32 + lane) * E;
    elems::Raw<DT, E> r[kEmbedFlight];
#pragma unroll
    for (int j = 0; j < kEmbedFlight; ++j) {
        const int64_t c = c0 + (int64_t)j * 32 * E;
        r[j].zero();
        if (row >= 0 && c < a.dim) r[j].load(a.table, row * a.table_stride + c);
    }
#pragma unroll
    for (int j = 0; j < kEmbedFlight; ++j) {
        const int64_t c = c0 + (int64_t)j * 32 * E;
        if (c >= a.dim) continue;
        if (row >= 0) {
            float f[E];
            r[j].get(f);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = __fmul_rn(f[e], a.scale);
            r[j].set(f);
        }
        r[j].store(a.out, i * a.out_stride + c);
    }
}

template <int DT, int E> cudaError_t embed_go(const EmbedArgs &a, cudaStream_t s)
{
    const int64_t per = (int64_t)32 * E * kEmbedFlight;
    const int64_t segs = (a.dim + per - 1) / per;
    const int64_t warps = a.tok.n * segs;
    // few rows: one warp a block, so that they spread over the SMs
    const int threads = warps <= 1024 ? 32 : kThreads;
    const int64_t blocks = (warps * 32 + threads - 1) / threads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(embed_kernel<DT, E>, dim3((unsigned)blocks), dim3((unsigned)threads),
                            0, s, a, (int)segs);
}

template <int DT> cudaError_t embed_pick(const EmbedArgs &a, cudaStream_t s)
{
    const int es = DT == F32 ? 4 : 2;
    const int e0 = row_access(a.table, a.table_stride, es, a.dim);
    const int e1 = row_access(a.out, a.out_stride, es, a.dim);
    const int e = e0 < e1 ? e0 : e1;
    return e == 8 ? embed_go<DT, 8>(a, s) : e == 2 ? embed_go<DT, 2>(a, s)
                                                   : embed_go<DT, 1>(a, s);
}

// ----------------------------------------------------------------- the sort
//
// A stable radix sort of (id, position) by 8-bit digits, lowest first; ids
// that name no row sort behind all rows.  Up to kSmallTokens tokens one block
// sorts in shared memory; beyond that every pass is two launches over
// at most 256 blocks: digit counts per block, then each block adds up the
// counts before its own and places its tokens.
constexpr int kSortThreads = 1024, kSortWarps = 32;
constexpr int kSmallTokens = 8192;
constexpr int kSortTile = 4096;
constexpr int kMaxSortBlocks = 256;

int sort_passes(int64_t rows)
{
    int p = 1;
    while (p < 4 && (rows >> (8 * p)) != 0) ++p;   // keys 0 .. rows (rows: names no row)
    return p;
}

int64_t sort_chunk(int64_t n)   // tokens per block of the multi-block sort
{
    const int64_t per = (n + kMaxSortBlocks - 1) / kMaxSortBlocks;
    return (per + kSortTile - 1) / kSortTile * kSortTile;
}

__device__ __forceinline__ uint32_t token_key(const TokenArgs &t, int64_t i)
{
    const int64_t row = token_row(t, i);
    return row < 0 ? (uint32_t)t.rows : (uint32_t)row;
}

// Lanes of the warp with the same digit (and `live`).
__device__ __forceinline__ uint32_t same_digit(uint32_t d, bool live)
{
    uint32_t m = __ballot_sync(0xffffffffu, live);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint32_t v = __ballot_sync(0xffffffffu, (d >> b) & 1);
        m &= ((d >> b) & 1) ? v : ~v;
    }
    return m;
}

// Exclusive prefix over the 32 warps of every digit's counts, in place; the
// digits' totals go to total[256].
__device__ __forceinline__ void prefix_warps(uint32_t (*count)[256], uint32_t *total)
{
    for (int d = threadIdx.x; d < 256; d += kSortThreads) {
        uint32_t run = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t v = count[w][d];
            count[w][d] = run;
            run += v;
        }
        total[d] = run;
    }
}

// Exclusive prefix of v[256] in place, by the first warp.
__device__ __forceinline__ void prefix_digits(uint32_t *v)
{
    if (threadIdx.x < 32) {
        uint32_t own[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            own[j] = v[threadIdx.x * 8 + j];
            sum += own[j];
        }
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if ((int)threadIdx.x >= o) inc += u;
        }
        uint32_t run = inc - sum;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[threadIdx.x * 8 + j] = run;
            run += own[j];
        }
    }
}

struct SmallSort {
    uint32_t count[kSortWarps][256];
    uint32_t total[256];
    uint32_t key[2][kSmallTokens];
    unsigned short idx[2][kSmallTokens];
};

// Zeroes rows of the gradient: `warps` warps of the grid, this one `warp`,
// a row each in turn; with `used`, only the rows that no token names.
template <int GT, int E>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs &a, const unsigned char *used,
                                          int64_t warp, int64_t warps)
{
    const int lane = threadIdx.x & 31;
    elems::Raw<GT, E> z;
    z.zero();
    for (int64_t r = warp; r < a.tok.rows; r += warps) {
        if (used && used[r]) continue;
        for (int64_t c = (int64_t)lane * E; c < a.dim; c += 32 * E)
            z.store(a.grad, r * a.grad_stride + c);
    }
}

// Block 0 sorts; the others zero the gradient meanwhile (unless it is added
// to): the rows that tokens name are written again afterwards, at most
// kSmallTokens of them, which costs less than the sort that it hides.
template <int GT, int E>
__global__ void __launch_bounds__(kSortThreads)
embed_sort_small_kernel(const __grid_constant__ EmbedGradArgs a, int passes)
{
    extern __shared__ __align__(16) unsigned char raw[];
    SmallSort &sm = *reinterpret_cast<SmallSort *>(raw);
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x != 0) {
        zero_rows<GT, E>(a, nullptr, (int64_t)(blockIdx.x - 1) * kSortWarps + warp,
                         (int64_t)(gridDim.x - 1) * kSortWarps);
        return;
    }
    const int n = (int)a.tok.n;
    if (threadIdx.x == 0) *a.n_runs = 0;
    const int iters = (n + kSortThreads - 1) / kSortThreads;     // <= 8
    for (int i = threadIdx.x; i < n; i += kSortThreads) {
        sm.key[0][i] = token_key(a.tok, i);
        sm.idx[0][i] = (unsigned short)i;
    }
    int from = 0;
    for (int p = 0; p < passes; ++p) {
        for (int i = threadIdx.x; i < kSortWarps * 256; i += kSortThreads)
            (&sm.count[0][0])[i] = 0;
        __syncthreads();
        uint32_t key[8], rank[8];
        unsigned short idx[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= iters) break;
            const int i = (warp * iters + j) * 32 + lane;
            const bool live = i < n;
            key[j] = live ? sm.key[from][i] : kNone;
            idx[j] = live ? sm.idx[from][i] : 0;
            const uint32_t d = (key[j] >> (8 * p)) & 255u;
            const uint32_t peers = same_digit(d, live);
            uint32_t before = 0;
            if (live) before = sm.count[warp][d];
            __syncwarp();
            rank[j] = before + __popc(peers & ((1u << lane) - 1));
            if (live && (peers >> lane) == 1u) sm.count[warp][d] = before + __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        prefix_warps(sm.count, sm.total);
        __syncthreads();
        prefix_digits(sm.total);
        __syncthreads();
        const int to = from ^ 1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= iters) break;
            const int i = (warp * iters + j) * 32 + lane;
            if (i < n) {
                const uint32_t d = (key[j] >> (8 * p)) & 255u;
                const uint32_t at = sm.total[d] + sm.count[warp][d] + rank[j];
                sm.key[to][at] = key[j];
                sm.idx[to][at] = idx[j];
            }
        }
        __syncthreads();
        from = to;
    }
    for (int i = threadIdx.x; i < n; i += kSortThreads) {
        a.key[0][i] = sm.key[from][i];
        a.idx[0][i] = sm.idx[from][i];
    }
}

// Digit counts of a block's tokens.  The first pass reads the tokens
// themselves, clears the map of used rows and the count of long runs.
__global__ void __launch_bounds__(kSortThreads)
embed_count_kernel(const __grid_constant__ EmbedGradArgs a, int pass, int64_t chunk)
{
    __shared__ uint32_t count[256];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t T = (int64_t)gridDim.x * kSortThreads;
    const int64_t t0 = (int64_t)blockIdx.x * kSortThreads + threadIdx.x;
    if (pass == 0) {
        if (t0 == 0) *a.n_runs = 0;
        for (int64_t r = t0; r < a.tok.rows; r += T) a.used[r] = 0;
    }
    if (threadIdx.x < 256) count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * chunk;
    const int64_t hi = lo + chunk < a.tok.n ? lo + chunk : a.tok.n;
    const uint32_t *key = a.key[(pass & 1) ^ 1];
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        const uint32_t k = pass == 0 ? token_key(a.tok, i) : key[i];
        atomicAdd(&count[(k >> (8 * pass)) & 255u], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 256) a.hist[blockIdx.x * 256 + threadIdx.x] = count[threadIdx.x];
}

// Pass `pass` reads side (pass & 1) ^ 1 (the tokens themselves at first) and
// writes side pass & 1.
__global__ void __launch_bounds__(kSortThreads)
embed_place_kernel(const __grid_constant__ EmbedGradArgs a, int pass, int64_t chunk)
{
    __shared__ uint32_t count[kSortWarps][256];
    __shared__ uint32_t total[256], base[256], part[4][2][256];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    {   // tokens of each digit in all blocks, and in the blocks before this one
        const int d = threadIdx.x & 255, quarter = threadIdx.x >> 8;
        uint32_t all = 0, before = 0;
#pragma unroll 8
        for (unsigned b = quarter; b < gridDim.x; b += 4) {
            const uint32_t v = a.hist[b * 256 + d];
            all += v;
            before += b < blockIdx.x ? v : 0u;
        }
        part[quarter][0][d] = all;
        part[quarter][1][d] = before;
    }
    __syncthreads();
    if (threadIdx.x < 256)
        total[threadIdx.x] = part[0][0][threadIdx.x] + part[1][0][threadIdx.x] +
                             part[2][0][threadIdx.x] + part[3][0][threadIdx.x];
    __syncthreads();
    prefix_digits(total);
    __syncthreads();
    if (threadIdx.x < 256)
        base[threadIdx.x] = total[threadIdx.x] + part[0][1][threadIdx.x] +
                            part[1][1][threadIdx.x] + part[2][1][threadIdx.x] +
                            part[3][1][threadIdx.x];
    const uint32_t *skey = a.key[(pass & 1) ^ 1], *sidx = a.idx[(pass & 1) ^ 1];
    uint32_t *dkey = a.key[pass & 1], *didx = a.idx[pass & 1];
    const int64_t lo = (int64_t)blockIdx.x * chunk;
    const int64_t hi = lo + chunk < a.tok.n ? lo + chunk : a.tok.n;
    constexpr int kIters = kSortTile / kSortThreads;
    for (int64_t tile = lo; tile < hi; tile += kSortTile) {
        for (int i = threadIdx.x; i < kSortWarps * 256; i += kSortThreads) (&count[0][0])[i] = 0;
        __syncthreads();
        uint32_t key[kIters], idx[kIters], rank[kIters];
#pragma unroll
        for (int j = 0; j < kIters; ++j) {
            const int64_t i = tile + (warp * kIters + j) * 32 + lane;
            const bool live = i < hi;
            key[j] = !live ? kNone : pass == 0 ? token_key(a.tok, i) : skey[i];
            idx[j] = !live ? 0u : pass == 0 ? (uint32_t)i : sidx[i];
        }
#pragma unroll
        for (int j = 0; j < kIters; ++j) {
            const bool live = tile + (warp * kIters + j) * 32 + lane < hi;
            if (pass == 0 && live && key[j] < (uint32_t)a.tok.rows) a.used[key[j]] = 1;
            const uint32_t d = (key[j] >> (8 * pass)) & 255u;
            const uint32_t peers = same_digit(d, live);
            uint32_t before = 0;
            if (live) before = count[warp][d];
            __syncwarp();
            rank[j] = before + __popc(peers & ((1u << lane) - 1));
            if (live && (peers >> lane) == 1u) count[warp][d] = before + __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        prefix_warps(count, total);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kIters; ++j) {
            if (tile + (warp * kIters + j) * 32 + lane < hi) {
                const uint32_t d = (key[j] >> (8 * pass)) & 255u;
                const uint32_t at = base[d] + count[warp][d] + rank[j];
                dkey[at] = key[j];
                didx[at] = idx[j];
            }
        }
        __syncthreads();
        if (threadIdx.x < 256) base[threadIdx.x] += total[threadIdx.x];
    }
}

// ------------------------------------------------------------------ the sums
//
// The sorted list is cut into chunks of C positions.  A warp takes a chunk
// and 256 columns, 8 a lane, and reads the chunk's rows of dy a few at a
// time.  A run of one id that lies within the chunk is finished there; one
// that passes an end of it leaves its fp32 part in the workspace (slot 0: the
// run that the chunk begins in the middle of, slot 1: the run that passes
// its end), and the chunk in which such a run begins enters it in a list
// whose entries embed_runs_kernel finishes.
constexpr int kCols = 256;

int64_t sum_chunk(int64_t n)
{
    int64_t c = 8;
    while (c < 256 && n > c * 4096) c *= 2;
    return c;
}

template <int YT, int GT, int E>
__device__ __forceinline__ void put_row(const EmbedGradArgs &a, uint32_t row, int64_t c0,
                                        const float (&acc)[8])
{
    constexpr int J = 8 / E;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int64_t c = c0 + (int64_t)j * 32 * E;
        if (c >= a.dim) continue;
        const int64_t at = (int64_t)row * a.grad_stride + c;
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = __fmul_rn(acc[j * E + e], a.scale);
        elems::Raw<GT, E> r;
        if (a.accumulate) {
            float o[E];
            r.load(a.grad, at);
            r.get(o);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = __fadd_rn(o[e], f[e]);
        }
        r.set(f);
        r.store(a.grad, at);
    }
}

// Both accesses of dy and of the gradient take E elements; lane `lane`'s
// element e of access j is column seg * 256 + j * 32 * E + lane * E + e.
template <int YT, int GT, int E>
__global__ void __launch_bounds__(kThreads)
embed_sum_kernel(const __grid_constant__ EmbedGradArgs a, int side, int64_t chunk, int segs,
                 int64_t sum_blocks)
{
    constexpr int J = 8 / E;
    constexpr int U = YT == F32 ? 4 : 8;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x >= sum_blocks) {
        zero_rows<GT, E>(a, a.used,
                         ((int64_t)(blockIdx.x - sum_blocks) * kThreads + threadIdx.x) >> 5,
                         ((int64_t)(gridDim.x - sum_blocks) * kThreads) >> 5);
        return;
    }
    const int64_t task = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int64_t ck = task / segs;
    const int seg = (int)(task - ck * segs);
    const int64_t lo = ck * chunk;
    if (lo >= a.tok.n) return;
    const int64_t hi = lo + chunk < a.tok.n ? lo + chunk : a.tok.n;
    const uint32_t *key = a.key[side], *idx = a.idx[side];
    const uint32_t none = (uint32_t)a.tok.rows;
    uint32_t cur = key[lo];
    if (cur == none) return;                      // sorted: nothing but such ids follows
    const uint32_t prev = lo > 0 ? key[lo - 1] : kNone;
    const uint32_t next = hi < a.tok.n ? key[hi] : kNone;
    const int64_t c0 = (int64_t)seg * kCols + lane * E;
    float *part = a.part + ck * 2 * (int64_t)segs * kCols + (int64_t)seg * kCols + lane * 8;
    bool begun = prev != cur;                     // the current run began in this chunk
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;

    auto flush = [&](bool ended) {
        if (begun && ended) {
            put_row<YT, GT, E>(a, cur, c0, acc);
        } else {
            float *p = part + (begun ? (int64_t)segs * kCols : 0);
            reinterpret_cast<float4 *>(p)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
            if (begun && seg == 0 && lane == 0) a.runs[atomicAdd(a.n_runs, 1u)] = (uint32_t)ck;
        }
    };

    for (int64_t base = lo; base < hi; base += 32) {
        const int m = (int)(hi - base < 32 ? hi - base : 32);
        const uint32_t mykey = lane < m ? key[base + lane] : none;
        const uint32_t myidx = lane < m ? idx[base + lane] : 0u;
        for (int u0 = 0; u0 < m; u0 += U) {
            elems::Raw<YT, E> r[U][J];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t k = __shfl_sync(0xffffffffu, mykey, (u0 + u) & 31);
                const uint32_t i = __shfl_sync(0xffffffffu, myidx, (u0 + u) & 31);
                const bool live = u0 + u < m && k != none;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int64_t c = c0 + (int64_t)j * 32 * E;
                    r[u][j].zero();
                    if (live && c < a.dim) r[u][j].load(a.dy, (int64_t)i * a.dy_stride + c);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t k = __shfl_sync(0xffffffffu, mykey, (u0 + u) & 31);
                if (u0 + u >= m || k == none) continue;
                if (k != cur) {
                    flush(true);
                    cur = k;
                    begun = true;
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float f[E];
                    r[u][j].get(f);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[j * E + e] = __fadd_rn(acc[j * E + e], f[e]);
                }
            }
        }
    }
    flush(next != cur);
}

// A block takes a listed run and 256 columns: its warps add up the parts
// they come to in turn, and the eight sums join in the warps' order.
template <int YT, int GT, int E>
__global__ void __launch_bounds__(kThreads)
embed_runs_kernel(const __grid_constant__ EmbedGradArgs a, int side, int64_t chunk, int segs)
{
    __shared__ float sums[8][kCols];
    __shared__ int64_t last_sh;
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tasks = (int64_t)*a.n_runs * segs;
    const uint32_t *key = a.key[side];
    for (int64_t t = blockIdx.x; t < tasks; t += gridDim.x) {
        const int64_t run = t / segs;
        const int seg = (int)(t - run * segs);
        const int64_t first = a.runs[run];
        const uint32_t id = key[(first + 1) * chunk];
        // the last chunk whose first id is the run's: 32 chunks at a time
        if (warp == 0) {
            int64_t last = first + 1;
            for (int64_t c = first + 1;; c += 32) {
                const int64_t at = (c + lane) * chunk;
                const uint32_t m = __ballot_sync(0xffffffffu, at < a.tok.n && key[at] == id);
                last = c + (m == 0xffffffffu ? 31 : __ffs(~m) - 2);
                if (m != 0xffffffffu) break;
            }
            if (lane == 0) last_sh = last;
        }
        __syncthreads();
        const int64_t last = last_sh;
        const int64_t step = 2 * (int64_t)segs * kCols;
        const float *p0 = a.part + (int64_t)seg * kCols + lane * 8;
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
#pragma unroll 4
        for (int64_t c = first + warp; c <= last; c += 8) {
            const float *p = p0 + c * step + (c == first ? (int64_t)segs * kCols : 0);
            const float4 u = reinterpret_cast<const float4 *>(p)[0];
            const float4 v = reinterpret_cast<const float4 *>(p)[1];
            acc[0] = __fadd_rn(acc[0], u.x);
            acc[1] = __fadd_rn(acc[1], u.y);
            acc[2] = __fadd_rn(acc[2], u.z);
            acc[3] = __fadd_rn(acc[3], u.w);
            acc[4] = __fadd_rn(acc[4], v.x);
            acc[5] = __fadd_rn(acc[5], v.y);
            acc[6] = __fadd_rn(acc[6], v.z);
            acc[7] = __fadd_rn(acc[7], v.w);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[warp][lane * 8 + e] = acc[e];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float s = sums[0][lane * 8 + e];
#pragma unroll
                for (int w = 1; w < 8; ++w) s = __fadd_rn(s, sums[w][lane * 8 + e]);
                acc[e] = s;
            }
            put_row<YT, GT, E>(a, id, (int64_t)seg * kCols + lane * E, acc);
        }
        __syncthreads();
    }
}

template <int YT, int GT, int E>
cudaError_t grad_go(const EmbedGradArgs &a, int sms, cudaStream_t s)
{
    const int64_t n = a.tok.n;
    const int passes = sort_passes(a.tok.rows);
    const bool small = n <= kSmallTokens;
    int side = 0;
    cudaError_t e;
    if (small) {
        static int attr_device = -1;   // the attribute is per device
        int dev = 0;
        cudaGetDevice(&dev);
        if (attr_device != dev) {
            e = cudaFuncSetAttribute(embed_sort_small_kernel<GT, E>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)sizeof(SmallSort));
            if (e != cudaSuccess) return e;
            attr_device = dev;
        }
        const unsigned blocks = a.accumulate ? 1u : (unsigned)(sms > 1 ? sms : 2);
        e = launch_dependent(embed_sort_small_kernel<GT, E>, dim3(blocks), dim3(kSortThreads),
                             sizeof(SmallSort), s, a, passes);
        if (e != cudaSuccess || n == 0) return e;
    } else {
        const int64_t chunk = sort_chunk(n);
        const unsigned blocks = (unsigned)((n + chunk - 1) / chunk);
        for (int p = 0; p < passes; ++p) {
            e = launch_dependent(embed_count_kernel, dim3(blocks), dim3(kSortThreads), 0, s, a, p,
                                 chunk);
            if (e != cudaSuccess) return e;
            e = launch_dependent(embed_place_kernel, dim3(blocks), dim3(kSortThreads), 0, s, a, p,
                                 chunk);
            if (e != cudaSuccess) return e;
        }
        side = (passes - 1) & 1;
    }
    const int64_t chunk = sum_chunk(n);
    const int segs = (int)((a.dim + kCols - 1) / kCols);
    const int64_t tasks = (n + chunk - 1) / chunk * segs;
    const int64_t sum_blocks = (tasks * 32 + kThreads - 1) / kThreads;
    const int64_t fill_blocks = !small && !a.accumulate ? (a.tok.rows + 63) / 64 : 0;
    if (sum_blocks + fill_blocks > 0x7fffffff) return cudaErrorInvalidValue;
    e = launch_dependent(embed_sum_kernel<YT, GT, E>, dim3((unsigned)(sum_blocks + fill_blocks)),
                         dim3(kThreads), 0, s, a, side, chunk, segs, sum_blocks);
    if (e != cudaSuccess) return e;
    const int64_t most = (n + chunk - 1) / chunk * segs;
    const int64_t grid = most < 4 * (int64_t)sms ? most : 4 * (int64_t)sms;
    return launch_dependent(embed_runs_kernel<YT, GT, E>, dim3((unsigned)grid), dim3(kThreads), 0,
                            s, a, side, chunk, segs);
}

template <int YT, int GT> cudaError_t grad_pick(const EmbedGradArgs &a, int sms, cudaStream_t s)
{
    const int e0 = row_access(a.dy, a.dy_stride, YT == F32 ? 4 : 2, a.dim);
    const int e1 = row_access(a.grad, a.grad_stride, GT == F32 ? 4 : 2, a.dim);
    const int e = e0 < e1 ? e0 : e1;
    return e == 8 ? grad_go<YT, GT, 8>(a, sms, s)
                  : e == 2 ? grad_go<YT, GT, 2>(a, sms, s) : grad_go<YT, GT, 1>(a, sms, s);
}

template <int YT>
cudaError_t grad_type(int32_t gdt, const EmbedGradArgs &a, int sms, cudaStream_t s)
{
    return gdt == F32 ? grad_pick<YT, F32>(a, sms, s)
                      : gdt == BF16 ? grad_pick<YT, BF16>(a, sms, s)
                                    : grad_pick<YT, F16>(a, sms, s);
}

}  // namespace

cudaError_t launch_embed(int32_t dt, const EmbedArgs &a, cudaStream_t s)
{
    if (a.tok.n <= 0 || a.dim <= 0) return cudaSuccess;
    return dt == F32 ? embed_pick<F32>(a, s) : dt == BF16 ? embed_pick<BF16>(a, s)
                                                          : embed_pick<F16>(a, s);
}

int64_t embed_grad_layout(EmbedGradArgs &a, char *base)
{
    const int64_t n = a.tok.n;
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        char *p = base + off;
        off += (bytes + 255) / 256 * 256;
        return p;
    };
    const int64_t chunks = (n + sum_chunk(n) - 1) / sum_chunk(n);
    const int64_t segs = (a.dim + kCols - 1) / kCols;
    a.n_runs = reinterpret_cast<uint32_t *>(take(4));
    a.runs = reinterpret_cast<uint32_t *>(take(4 * chunks));
    for (int i = 0; i < 2; ++i) {
        // one block sorts a short list in shared memory: one side is enough
        const int64_t len = i == 1 && n <= kSmallTokens ? 0 : n;
        a.key[i] = reinterpret_cast<uint32_t *>(take(4 * len));
        a.idx[i] = reinterpret_cast<uint32_t *>(take(4 * len));
    }
    const bool big = n > kSmallTokens;
    a.hist = reinterpret_cast<uint32_t *>(take(big ? 4 * 256 * kMaxSortBlocks : 0));
    a.used = reinterpret_cast<unsigned char *>(take(big ? a.tok.rows : 0));
    a.part = reinterpret_cast<float *>(take(chunks * 2 * segs * kCols * 4));
    return off > 0 ? off : 256;
}

cudaError_t launch_embed_grad(int32_t ydt, int32_t gdt, const EmbedGradArgs &a, int sms,
                              cudaStream_t s)
{
    if (a.dim <= 0 || a.tok.rows <= 0) return cudaSuccess;
    if (a.tok.n <= 0 && a.accumulate) return cudaSuccess;
    return ydt == F32 ? grad_type<F32>(gdt, a, sms, s)
                      : ydt == BF16 ? grad_type<BF16>(gdt, a, sms, s)
                                    : grad_type<F16>(gdt, a, sms, s);
}

}  // namespace zgb
